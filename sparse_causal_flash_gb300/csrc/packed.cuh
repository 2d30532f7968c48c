// Attention over packed sequences with shared key heads: what the plan, the forward and the backward have in common.
//
// A tile of query rows is TPT = 128 / G tokens times the G query heads of one key head, row (token, head of the group)
// at token * G + head: the heads that share keys share every key tile that is loaded, and a causal border inside a
// tile is TPT tokens wide instead of 128. (G = 3: 42 tokens, 126 rows; the rows behind stay zero in shared memory.)
// A tile of keys is 128 keys of one sequence. The plan cuts the work of one key head into entries; a kernel's work item
// w is entry w / Hkv for key head w % Hkv.
#pragma once

#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"

namespace scfa {

constexpr uint32_t kPackMagic = 0x50414b31u;
constexpr int kPackSub = kTile * 128;  // bytes of a [128 rows][64 channels] swizzled sub-tile
constexpr float kPackLog2e = 1.4426950408889634f;
constexpr float kPackLn2 = 0.6931471805599453f;
// Chunks that cut entries may leave behind for their join, over all key heads.
constexpr int kPackSlotsPerSm = 4;

// Work of so many tiles is never cut, so that calls on few rows need no join (7 short texts, in a graph:
// 9.4 us instead of 10.8 forward, 16.8 instead of 19.0 backward; other numbers were not measured). What is cut depends on the
// longest range of a tile, which the host does not know: it goes by the rows of the whole call, and larger calls that are
// not cut either have an empty join behind them (2 to 3.5 us).
constexpr int kPackNeverCut = 3;
inline bool pack_may_cut(int N, int M, int tpt, bool backward) {
  return M > kPackNeverCut * kTile || (backward && N > kPackNeverCut * tpt);
}

enum { kListFwd = 0, kListDq = 1, kListDkv = 2, kLists = 3 };

// One piece of work of one key head. Query lists: the tokens q0 .. q0 + n_tok (rows of q) see the keys k0 .. of one
// sequence; token i sees the sequence's keys up to diag + i, and in this entry tiles [a, b) of them. Key list: the keys
// k0 .. k0 + n_tok (rows of k; at `diag` in their sequence) with the query tiles [a, b) of the sequence, whose tokens
// start at row q0; token t sees the keys up to t + shift.
struct PackEntry {
  int q0, k0, n_tok, diag;
  int a, b;
  int m;       // query lists: keys of the sequence. Key list: its tokens
  int shift;   // key list: keys minus queries of the sequence
  int tile0;   // number of the (first) query tile over all sequences
  int slot;    // first partial slot of the cut entry (per key head); -1: not cut
  int chunk, chunks;
  int head;    // (in shared memory) key head, -1: no more work
  int seq;     // number of the sequence
  int pad[2];
};
static_assert(sizeof(PackEntry) == 64, "entries are copied as 16 words");

struct PackHeader {
  int status;  // SCFA_OK or what is wrong with the sequences
  int rows;    // (at byte 4, as the interface says) where the last sequence's queries end; 0 for a batch that is refused
  uint32_t magic;
  int N, M, R, Hq, Hkv, window;
  int n_entries[kLists];
  int n_qtiles;            // query tiles of all sequences
  int list_status[kLists];  // (each list is built by a CTA of its own)
  int n_cuts[kLists];       // entries that are cut, per key head
  int pad0[2];
  long long entries[kLists];  // byte offsets from the plan's start
  long long cuts[kLists];     // PackEntry: the first chunk of each cut one
  long long qtiles;           // int4 (first token, tokens, last key of the first token, 0) of each query tile
  long long bytes;
  int pad[26];
};
static_assert(sizeof(PackHeader) == 256, "the plan's header");

struct PackPlanLayout {
  // first tile of each sequence [kLists + 1][R + 1] (the last one: query tiles again, for the key list's CTA); (units,
  // sequence) of each tile, list by list; the rest is what the header names
  size_t pre = 0, units[kLists] = {}, qtiles = 0, entries[kLists] = {}, cuts[kLists] = {}, total = 0;
  long long most[kLists] = {};  // entries of each list at most
};

inline int pack_slots(int sms) { return kPackSlotsPerSm * sms; }

// false if the sizes are out of range
inline bool pack_plan_layout(int N, int M, int R, int Hq, int Hkv, int sms, PackPlanLayout* L) {
  if (N < 0 || M < 0 || R < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > kTile) return false;
  const int tpt = kTile / (Hq / Hkv);
  PackPlanLayout w;
  const long long extra = static_cast<long long>(R) + pack_slots(sms);
  w.most[kListFwd] = N / (2 * tpt) + extra;
  w.most[kListDq] = N / tpt + extra;
  w.most[kListDkv] = M / kTile + extra;
  for (long long n : w.most)
    if (n * Hkv >= (1ll << 31) - 1024) return false;
  size_t off = sizeof(PackHeader);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  w.pre = take(static_cast<size_t>(kLists + 1) * (R + 1) * sizeof(int));
  for (int i = 0; i < kLists; ++i) w.units[i] = take(static_cast<size_t>(w.most[i]) * sizeof(int2));
  w.qtiles = take((static_cast<size_t>(N / tpt) + R) * sizeof(int4));
  for (int i = 0; i < kLists; ++i) w.entries[i] = take(static_cast<size_t>(w.most[i]) * sizeof(PackEntry));
  for (int i = 0; i < kLists; ++i) w.cuts[i] = take(static_cast<size_t>(pack_slots(sms)) / 2 * sizeof(PackEntry));
  w.total = off;
  *L = w;
  return true;
}

// Workspace: status and work counters, then the chunks' partial results, then (backward) the rows' statistics.
struct PackWs {
  size_t counters = 0;          // ints: next item of each kernel
  size_t part = 0, part_q = 0;  // fp32, [slot][Hkv]: two tiles of D + 2 columns, or dV and dK; (backward) dQ
  size_t forward = 0;           // what a forward needs
  size_t stats = 0;             // backward: [2][query tiles][Hkv][128] floats, then for fp16 lengths of rows (packed_bwd.cu):
                                // [query tiles][Hkv][128] and [..][16] of dO, [key tiles][Hkv][8] of V
  size_t clear = 0;             // bytes from the start that a call clears
};
// A backward's workspace serves a forward too.
inline PackWs pack_ws(int D, int sms) {
  PackWs w;
  const size_t slots = static_cast<size_t>(pack_slots(sms)), row = static_cast<size_t>(kTile) * sizeof(float);
  w.counters = sizeof(WsHeader);
  w.clear = w.part = align_up(w.counters + 2 * sizeof(int), 256);
  w.forward = align_up(w.part + slots * 2 * row * (D + 2), 256);
  w.part_q = align_up(w.part + slots * 2 * row * D, 256);
  w.stats = align_up(w.part_q + slots * row * D, 256);
  return w;
}
constexpr int kDoUnits = 16, kVUnits = 8;  // a tile's pieces of 8 and 16 rows
__host__ __device__ __forceinline__ long long pack_stats_bytes(long long q_tiles, int M, int R, int Hkv) {
  return (q_tiles * (3 * kTile + kDoUnits) + (static_cast<long long>(M / kTile) + R) * kVUnits) * Hkv * static_cast<long long>(sizeof(float));
}
// Number of key tile i (of the sequence seq, whose keys start at row k0) among less than M / 128 + R: sequences of m keys
// leave room for as many tiles as they may have.
__device__ __forceinline__ long long pack_key_tile(int k0, int seq, int i) { return static_cast<long long>(k0 / kTile) + seq + i; }

// The join of what the chunks left, behind the kernel that left it: o and lse (forward), or dV, dK and dQ.
struct PackJoin {
  const char* plan;
  long long plan_bytes;
  int N, M, Hq, Hkv, G, tpt;
  const float *part, *part_q;
  float scale;
  uint16_t *o, *dq, *dk, *dv;
  long long ot, oh, dqt, dqh, dkt, dkh, dvt, dvh;
  float* lse;
  const int* status;
};
cudaError_t launch_pack_join(const PackJoin& j, int D, bool f16, bool backward, int sms, cudaStream_t st);

// What every kernel checks first: the plan is one for this call and lies in its buffer.
__device__ __forceinline__ int pack_plan_status(const PackHeader* h, long long bytes, int N, int M, int Hq, int Hkv) {
  if (h->magic != kPackMagic || h->N != N || h->M != M || h->Hq != Hq || h->Hkv != Hkv || h->bytes > bytes) return SCFA_ERR_INVALID;
  for (int i = 0; i < kLists; ++i)
    if (h->list_status[i] != SCFA_OK) return h->list_status[i];
  return SCFA_OK;
}

// instruction descriptor of kind::f16 with fp32 accumulators, both operands bf16 or both fp16
template <bool F16>
__host__ __device__ constexpr uint32_t pack_idesc(int M, int N, int a_mn, int b_mn) {
  return F16 ? (idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10))) : idesc_bf16_f32(M, N, a_mn, b_mn);
}

// One lane of a whole warp, by the instruction that the compiler knows as such: code under it may keep its operands in
// uniform registers, as MMAs want them (under `lane == 0` issuing was what bounded
// the forward: 517 us instead of 440 at 8192 tokens, 32 heads over 8 of 128 channels, at that stage).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// MMAs whose operands lie at a fixed distance (OFF, in 16-byte units) from a descriptor of which only the low word
// changes: the distance is added inside, so that one word per operand is all that has to reach the uniform registers.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024 bytes, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | (((lbo_bytes >> 4) & 0x3FFFu) << 16);
}
template <int A_OFF, int B_OFF>
__device__ __forceinline__ void mma_ss_at(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\tmov.b64 a, {x, %7};\n\tmov.b64 b, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(A_OFF), "n"(B_OFF), "n"(kDescHigh) : "memory");
}
// A in tensor memory, A_COL columns from a_tmem
template <int A_COL, int B_OFF>
__device__ __forceinline__ void mma_ts_at(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\tmov.b64 b, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(A_COL), "n"(B_OFF), "n"(kDescHigh) : "memory");
}
// Steps KK .. END of a product over K-major operands in shared memory (64-channel sub-tiles), 16 channels a step.
template <int KK, int END>
__device__ __forceinline__ void mma_ss_steps(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool add_to) {
  if constexpr (KK < END) {
    constexpr int off = static_cast<int>(kstep_off16(KK, kPackSub));
    mma_ss_at<off, off>(d_tmem, a_low, b_low, idesc, KK > 0 || add_to ? 1u : 0u);
    mma_ss_steps<KK + 1, END>(d_tmem, a_low, b_low, idesc, add_to);
  }
}
// Steps KK .. END of a product whose A (16 bits, K pairs along the columns) is in tensor memory and whose B has its rows
// along K in shared memory, 16 rows a step; `steps` of all of them hold something.
template <int KK, int END>
__device__ __forceinline__ void mma_ts_steps(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool add_to, int steps) {
  if constexpr (KK < END) {
    if (KK < steps) mma_ts_at<KK * 8, KK * 128>(d_tmem, a_tmem, b_low, idesc, KK > 0 || add_to ? 1u : 0u);
    mma_ts_steps<KK + 1, END>(d_tmem, a_tmem, b_low, idesc, add_to, steps);
  }
}

// one arrival for a warp, behind all its lanes' work
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// a wait by a whole warp (false for every lane if one gave up). The usual case is one vote that all lanes leave by together:
// with lanes returning one by one a wait that is over already cost 60 cycles more (1253 -> 1224 us forward at 16384 tokens,
// 32 heads over 8 of 128 channels).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}

// 16 lanes x 32 columns: r[4 i + 2 u + v] is lane (lane / 4 + 8 u), column 8 i + 2 (lane % 4) + v
__device__ __forceinline__ void tmem_ld_quad(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// use(c, words) for 16 lanes of an accumulator of W columns, 32 columns (from c) at a time, the next ones on their way;
// zeros without `some`. A loop, and a short one: code that runs once an item is fetched anew each time (unrolled, the
// forward of 8192 tokens, 32 heads over 8 of 128 channels took 346 us instead of 338).
template <int W, typename Use>
__device__ __forceinline__ void quad_blocks(uint32_t taddr, bool some, Use use) {
  uint32_t next[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) next[i] = 0u;
  if (some) tmem_ld_quad(taddr, next);
#pragma unroll 1
  for (int c = 0; c < W; c += 32) {
    uint32_t acc[16];
    if (some) {
      tmem_wait_ld();
      tmem_ld_fence(next);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = next[i];
    if (some && c + 32 < W) tmem_ld_quad(taddr + c + 32, next);
    use(c, acc);
  }
}
// All W columns of 16 lanes at once.
template <int W>
__device__ __forceinline__ void quad_part(uint32_t taddr, bool some, uint32_t (&acc)[W / 32][16]) {
#pragma unroll
  for (int b = 0; b < W / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[b][i] = 0u;
  if (some) {
#pragma unroll
    for (int b = 0; b < W / 32; ++b) tmem_ld_quad(taddr + 32 * b, acc[b]);
    tmem_wait_ld();
#pragma unroll
    for (int b = 0; b < W / 32; ++b) tmem_ld_fence(acc[b]);
  }
}
// One of the two rows that a quad of lanes holds (u), times f, in the rows' type to `row`: 32 channels. Four words change
// places inside the quad so that each lane has 16 bytes and the quad 64 in a row: a quarter of the stores' lines that whole
// rows per thread would touch (those took 6,500 cycles for a tile of 128 x 128).
template <bool F16>
__device__ __forceinline__ void quad_store(uint16_t* row, bool live, const uint32_t (&acc)[16], int u, float f) {
  const int t = threadIdx.x & 3;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = c4_pack<F16>(__uint_as_float(acc[i * 4 + 2 * u]) * f, __uint_as_float(acc[i * 4 + 2 * u + 1]) * f);
  const uint32_t x0 = __shfl_xor_sync(0xffffffffu, t & 1 ? w[0] : w[1], 1), x1 = __shfl_xor_sync(0xffffffffu, t & 1 ? w[2] : w[3], 1);
  const uint32_t p0 = t & 1 ? x0 : w[0], p1 = t & 1 ? w[1] : x0, p2 = t & 1 ? x1 : w[2], p3 = t & 1 ? w[3] : x1;
  const uint32_t y0 = __shfl_xor_sync(0xffffffffu, t & 2 ? p0 : p2, 2), y1 = __shfl_xor_sync(0xffffffffu, t & 2 ? p1 : p3, 2);
  const uint4 v = t & 2 ? make_uint4(y0, y1, p2, p3) : make_uint4(p0, p1, y0, y1);
  if (live) *reinterpret_cast<uint4*>(row + 8 * t) = v;
}
// Leave 32 columns of an accumulator (rows of D) as a chunk's share; TIMES: the quad's two rows times f.
template <int D, bool TIMES = false>
__device__ __forceinline__ void leave_part(float* mine, const uint32_t (&acc)[16], int row, const float (&f)[2] = {}) {
  const int c0 = 2 * (threadIdx.x & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<float2*>(mine + (row + 8 * u) * D + 8 * i + c0) =
          make_float2(__uint_as_float(acc[i * 4 + 2 * u]) * (TIMES ? f[u] : 1.f), __uint_as_float(acc[i * 4 + 2 * u + 1]) * (TIMES ? f[u] : 1.f));
}
// The largest of three, one instruction. Scores from TMEM pass tmem_ld_fence() before they come here: to the compiler they are
// there as soon as their load is issued, and it may put this asm above the wait for it.
__device__ __forceinline__ float pack_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Bits from .. to - 1 of 32, either end anywhere.
__device__ __forceinline__ uint32_t bit_range(int from, int to) {
  from = max(from, 0), to = min(to, 32);
  return from < to ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
}
// Bits c and c + 1 as a mask of two 16-bit values.
__device__ __forceinline__ uint32_t bit_pair(uint32_t bits, int c) {
  return (bits >> c & 1u ? 0x0000ffffu : 0u) | (bits >> (c + 1) & 1u ? 0xffff0000u : 0u);
}

// launch_behind() with shared memory; `behind` false: an ordinary launch.
template <typename... Params, typename... Args>
cudaError_t launch_behind_with(void (*kern)(Params...), dim3 grid, int threads, size_t smem, bool behind, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Registers of a warpgroup's threads, which all of its warps change together: fewer, or more of what others gave up.
template <int N>
__device__ __forceinline__ void regs_release() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }

// The producer warp's way to its pieces of work: the CTA's first one by its number, fetched while the CTA is set up, the
// others from the counter, one ahead.
struct PackWork {
  const PackEntry* entries;
  int n_work, Hkv, w, word;
  __device__ __forceinline__ void fetch(int lane) {
    word = w < n_work && lane < 16 ? __ldg(reinterpret_cast<const int*>(entries + w / Hkv) + lane) : 0;
  }
  __device__ __forceinline__ void first(const PackEntry* e, int n, int heads, int lane) {
    entries = e, n_work = n, Hkv = heads, w = static_cast<int>(blockIdx.x);
    fetch(lane);
  }
  __device__ __forceinline__ void next(int* counter, int lane) {
    int v = 0;
    if (lane == 0) v = atomicAdd(counter, 1);
    w = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, v, 0);
    fetch(lane);
  }
  // the piece into its slot; false at the end
  __device__ __forceinline__ bool publish(PackEntry* slot, uint64_t* full, int lane) {
    const bool some = w < n_work;
    if (some && lane < 16) reinterpret_cast<int*>(slot)[lane] = word;
    __syncwarp();
    if (lane == 0) slot->head = some ? w % Hkv : -1;
    warp_arrive(full);
    return some;
  }
};

// Rows [from, to) of a tile in shared memory become zero (whole rows: the swizzle moves 16-byte pieces inside a row).
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int subs, int from, int to, int lane, int lanes) {
  for (int i = lane; i < (to - from) * 8 * subs; i += lanes) {
    const int sub = i / ((to - from) * 8), at = i % ((to - from) * 8);
    *reinterpret_cast<uint4*>(tile + sub * kPackSub + from * 128 + at * 16) = make_uint4(0, 0, 0, 0);
  }
}

// 3-D map {channels, heads, tokens} over rows with their own strides (in elements); box = 64 channels x `box_heads`
// heads x `box_tokens` tokens, 128-byte swizzle, zeros behind the ends.
bool make_tmap_rows(CUtensorMap* map, const void* base, bool f16, int D, int heads, long long tokens, long long head_stride,
                    long long token_stride, int box_heads, int box_tokens);

// A read operand of the packed calls: aligned, with positive strides where an axis is longer than one.
inline bool pack_rows_ok(const void* p, long long token, long long head, long long N, int H) {
  if (!p || (reinterpret_cast<uintptr_t>(p) & 15u) || ((token | head) & 7)) return false;
  return (N <= 1 || (token > 0 && token < (1ll << 38))) && (H <= 1 || (head > 0 && head < (1ll << 38)));
}

}  // namespace scfa
