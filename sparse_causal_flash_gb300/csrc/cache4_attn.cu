// Attention of new tokens over the paged 4-bit cache.
#include <climits>

#include "cache4.cuh"
#include "internal.h"

namespace scfa {
namespace {

struct C4AttnArgs {
  const uint16_t* q;
  long long qt, qh;
  const uint8_t* cache;
  int page_size, n_pages;
  const int32_t* table;
  int max_pages;
  const int32_t *q_start, *vis;
  int N, R, Hq, Hkv;
  float scale;
  uint16_t* o;
  long long ot, oh;
  float* lse;
  int* status;
};

// One CTA per (token, query head), 128 keys at a time: thread = key for the
// scores, thread = channel for the values.
template <int D, bool F16>
__global__ void __launch_bounds__(128) attn_simple_kernel(C4AttnArgs a) {
  using L = C4<D>;
  __shared__ float sq[D], sp[128], red[4];
  __shared__ long long sbase[128];
  const int tok = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hkv), tid = threadIdx.x;
  if (tok >= a.q_start[a.R]) return;
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  const int vis = static_cast<int>(min(cap, static_cast<long long>(max(0, a.vis[tok]))));
  if (tid < D / 2) {
    const float2 f = c4_unpack<F16>(reinterpret_cast<const uint32_t*>(a.q + tok * a.qt + h * a.qh)[tid]);
    sq[2 * tid] = f.x, sq[2 * tid + 1] = f.y;
  }
  float m = -INFINITY, l = 0.f, o = 0.f;
  __syncthreads();
  for (int p0 = 0; p0 < vis; p0 += 128) {
    const int pos = p0 + tid;
    float s = -INFINITY;
    sbase[tid] = -1;
    if (pos < vis) {
      const int page = a.table[static_cast<long long>(lo) * a.max_pages + pos / a.page_size];
      if (page >= 0 && page < a.n_pages) {
        const int at = pos % a.page_size, t = at & 15;
        sbase[tid] = c4_tile_base(page, a.Hkv, hk, a.page_size, at, L::kTileBytes);
        const uint8_t* tile = a.cache + sbase[tid];
        s = 0.f;
        for (int g = 0; g < L::kG; ++g) {
          float x = 0.f;
          for (int j = 0; j < 4; ++j) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(tile + L::k_row(t) + (j * L::kG + g) * 4);
            for (int y = 0; y < 8; ++y)
              x += sq[32 * g + 8 * j + (y < 4 ? 2 * y : 2 * y - 7)] *
                   static_cast<float>(static_cast<int>(c >> (4 * y) & 15u) - 8);
          }
          s += x * c4_scale(tile[L::kKScales + t * L::kG + g]);
        }
        s *= a.scale;
      } else {
        raise_status(a.status, SCFA_ERR_INVALID);
      }
    }
    float x = s;
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    if ((tid & 31) == 0) red[tid >> 5] = x;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - base);
    sp[tid] = expf(s - base);
    __syncthreads();
    l *= f, o *= f, m = mn;
    const int r = tid % 32 / 4, y = tid % 4, g = tid / 32;
    for (int k = 0; k < 128; ++k) {
      l += sp[k];
      if (tid < D && sbase[k] >= 0) {
        const uint8_t* tile = a.cache + sbase[k];
        const int t = (p0 + k) & 15;
        const uint32_t c = *reinterpret_cast<const uint16_t*>(tile + L::v_piece(t, r) + 2 * g);
        o += sp[k] * static_cast<float>(static_cast<int>(c >> (4 * y) & 15u) - 8) *
             c4_scale(tile[L::kVScales + t * L::kG + g]);
      }
    }
    __syncthreads();
  }
  if (tid < D) {
    const float v = l > 0.f ? o / l : 0.f;
    a.o[tok * a.ot + h * a.oh + tid] = static_cast<uint16_t>(c4_pack<F16>(v, 0.f) & 0xFFFFu);
  }
  if (tid == 0) a.lse[static_cast<long long>(tok) * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

__global__ void clear_status_kernel(int* status) { *status = SCFA_OK; }

}  // namespace
}  // namespace scfa

using namespace scfa;

extern "C" {

size_t scfa_cache4_attn_workspace_size(int N, int R, int Hq, int Hkv, int D) {
  if (N < 1 || R < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return sizeof(WsHeader);
}

scfa_status scfa_cache4_attn(const uint16_t* q, long long q_token, long long q_head, const uint8_t* cache,
                             int page_size, int n_pages, const int32_t* table, int max_pages,
                             const int32_t* q_start, const int32_t* vis, int N, int R, int Hq, int Hkv, int D,
                             float scale, int dtype, uint16_t* o, long long o_token, long long o_head, float* lse,
                             void* ws, size_t ws_bytes, unsigned flags, void* stream) {
  if (!q || !cache || !table || !q_start || !vis || !o || !lse || !ws) return SCFA_ERR_INVALID;
  if (N < 1 || R < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || n_pages < 1 || max_pages < 1) return SCFA_ERR_INVALID;
  if (!(scale > 0.f && scale < INFINITY)) return SCFA_ERR_INVALID;
  if (dtype != SCFA_DTYPE_BF16 && dtype != SCFA_DTYPE_F16) return SCFA_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || !c4_page_size_ok(page_size)) return SCFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_pages) * page_size >= (1ll << 31) ||
      static_cast<long long>(max_pages) * page_size >= (1ll << 31))
    return SCFA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(q), static_cast<const void*>(cache), static_cast<const void*>(o)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SCFA_ERR_INVALID;
  if ((q_token | q_head | o_token | o_head) & 7) return SCFA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < scfa_cache4_attn_workspace_size(N, R, Hq, Hkv, D))
    return SCFA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const C4AttnArgs a = {q, q_token, q_head, cache, page_size, n_pages, table, max_pages, q_start, vis, N, R, Hq, Hkv,
                        scale, o, o_token, o_head, lse, static_cast<int*>(ws)};
  clear_status_kernel<<<1, 1, 0, st>>>(a.status);
  const bool f = dtype == SCFA_DTYPE_F16;
  auto kern = D == 64 ? (f ? attn_simple_kernel<64, true> : attn_simple_kernel<64, false>)
                      : (f ? attn_simple_kernel<128, true> : attn_simple_kernel<128, false>);
  if (static_cast<long long>(N) * Hq > INT_MAX) return SCFA_ERR_UNSUPPORTED;
  kern<<<N * Hq, 128, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SCFA_ERR_CUDA;
  if ((flags & SCFA_FLAG_DEBUG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return SCFA_ERR_CUDA;
  return SCFA_OK;
}

}  // extern "C"
