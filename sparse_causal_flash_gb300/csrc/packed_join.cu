// Joins what chunks of cut work left behind (packed_plan.cu): one row by a warp (128 channels) or half a warp (64), its
// chunks in their order, so that results are the same bits on every run. Bounded by L2: every share is read once (12 us,
// alone and with cold caches, for the 17 MB of three chunks over 12,000 keys). The last chunk to arrive joining for all
// took 27 us for eight chunks on its one SM, at the end of the kernel.
#include "packed.cuh"

namespace scfa {
namespace {

constexpr int kJoinThreads = 256, kAhead = 4;

__device__ __forceinline__ void add4(float4& a, float4 x, float f) {
  a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y), a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
}
template <bool F16>
__device__ __forceinline__ void put4(uint16_t* dst, float4 a, float f) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(c4_pack<F16>(a.x * f, a.y * f), c4_pack<F16>(a.z * f, a.w * f));
}

template <int D, bool F16, bool BACK>
__global__ void __launch_bounds__(kJoinThreads) packed_join_kernel(const __grid_constant__ PackJoin j) {
  constexpr int L = D / 4;  // lanes of a row
  grid_wait();  // (the shares of a kernel two before, and the status, are read past L1)
  const PackHeader* const h = reinterpret_cast<const PackHeader*>(j.plan);
  if (pack_plan_status(h, j.plan_bytes, j.N, j.M, j.Hq, j.Hkv) != SCFA_OK || __ldcg(j.status) != SCFA_OK) return;
  const int lane = threadIdx.x % L;
  const uint32_t step = gridDim.x * (kJoinThreads / L), first = blockIdx.x * (kJoinThreads / L) + threadIdx.x / L;
#pragma unroll 1
  for (int list = BACK ? kListDq : kListFwd; list <= (BACK ? kListDkv : kListFwd); ++list) {
    const PackEntry* const cuts = reinterpret_cast<const PackEntry*>(j.plan + h->cuts[list]);
    const uint32_t tiles = list == kListDq ? 1 : 2;  // two query tiles, or dV and dK
    const uint32_t rows = static_cast<uint32_t>(h->n_cuts[list]) * j.Hkv * tiles * kTile;  // (cuts x heads: half the slots)
    for (uint32_t i = first; i < rows; i += step) {
      const int r = static_cast<int>(i % kTile), x = static_cast<int>(i / kTile % tiles);
      const int head = static_cast<int>(i / (kTile * tiles) % static_cast<uint32_t>(j.Hkv));
      const PackEntry& e = cuts[i / (kTile * tiles * static_cast<uint32_t>(j.Hkv))];
      const int n_tok = __ldg(&e.n_tok), n = __ldg(&e.chunks), slot = __ldg(&e.slot), q0 = __ldg(&e.q0), k0 = __ldg(&e.k0);
      const int tok = list == kListDkv ? r : x * j.tpt * (list == kListFwd) + r / j.G;
      if (tok >= n_tok || (list != kListDkv && r >= j.G * j.tpt)) continue;
      constexpr int cols = D + (BACK ? 0 : 2);
      const long long stride = static_cast<long long>(j.Hkv) * tiles * kTile * cols;  // from chunk to chunk
      const float* const base = (list == kListDq ? j.part_q : j.part) +
          ((static_cast<long long>(slot) * j.Hkv + head) * tiles + x) * kTile * cols;
      const float4* const mine = reinterpret_cast<const float4*>(base + r * D) + lane;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!BACK) {
        const float2* const ml = reinterpret_cast<const float2*>(base + kTile * D) + r;
        float m = -INFINITY, l = 0.f;
        for (int c0 = 0; c0 < n; c0 += kAhead) {  // sums and shares of a few chunks in flight
          float2 z[kAhead];
          float4 y[kAhead];
#pragma unroll
          for (int c = 0; c < kAhead; ++c) {
            const int at = min(c0 + c, n - 1);
            z[c] = __ldcg(ml + at * (stride / 2));
            y[c] = __ldcg(mine + at * (stride / 4));
          }
          float top = m;
#pragma unroll
          for (int c = 0; c < kAhead; ++c) top = fmaxf(top, z[c].x);
          const float was = m == -INFINITY ? 0.f : ex2_approx(m - top);
          l *= was, acc.x *= was, acc.y *= was, acc.z *= was, acc.w *= was;
          m = top;
#pragma unroll
          for (int c = 0; c < kAhead; ++c) {
            if (c0 + c >= n) break;
            // a chunk in which the row sees nothing weighs nothing; NaN stays NaN
            const float f = z[c].x == -INFINITY ? (z[c].y == z[c].y ? 0.f : z[c].y) : ex2_approx(z[c].x - m);
            l = fmaf(z[c].y, f, l);
            add4(acc, y[c], f);
          }
        }
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        const long long t = static_cast<long long>(q0) + tok;
        const int qh = head * j.G + r % j.G;
        put4<F16>(j.o + t * j.ot + qh * j.oh + 4 * lane, acc, inv);
        if (lane == 0) j.lse[t * j.Hq + qh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kPackLn2;
      } else {
        for (int c0 = 0; c0 < n; c0 += kAhead) {
          float4 y[kAhead];
#pragma unroll
          for (int c = 0; c < kAhead; ++c) y[c] = __ldcg(mine + min(c0 + c, n - 1) * (stride / 4));
#pragma unroll
          for (int c = 0; c < kAhead; ++c)
            if (c0 + c < n) add4(acc, y[c], 1.f);
        }
        if (list == kListDq)
          put4<F16>(j.dq + static_cast<long long>(q0 + tok) * j.dqt + (head * j.G + r % j.G) * j.dqh + 4 * lane, acc, j.scale);
        else if (x)
          put4<F16>(j.dk + static_cast<long long>(k0 + tok) * j.dkt + head * j.dkh + 4 * lane, acc, j.scale);
        else
          put4<F16>(j.dv + static_cast<long long>(k0 + tok) * j.dvt + head * j.dvh + 4 * lane, acc, 1.f);
      }
    }
  }
}

template <int D, bool F16>
cudaError_t launch(const PackJoin& j, bool backward, int sms, cudaStream_t st) {
  return backward ? launch_behind(packed_join_kernel<D, F16, true>, dim3(4 * sms), kJoinThreads, st, j)
                  : launch_behind(packed_join_kernel<D, F16, false>, dim3(4 * sms), kJoinThreads, st, j);
}

}  // namespace

cudaError_t launch_pack_join(const PackJoin& j, int D, bool f16, bool backward, int sms, cudaStream_t st) {
  return D == 64 ? (f16 ? launch<64, true>(j, backward, sms, st) : launch<64, false>(j, backward, sms, st))
                 : (f16 ? launch<128, true>(j, backward, sms, st) : launch<128, false>(j, backward, sms, st));
}

}  // namespace scfa
