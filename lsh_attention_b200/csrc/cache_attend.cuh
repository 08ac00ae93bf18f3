// Shared-QK attention of a sequence's newest tokens over the paged cache.
//
// Row t at position p = len + t sees the cached tokens j <= p:
//   l_j = x_t . k_j / (||x_j|| sqrt(d)),  l_p = -1e5,
//   out = sum_j softmax(l)_j v_j,  lse = ln sum_j exp l_j.
#pragma once

#include "cache.cuh"

namespace lsh {

struct AttendArgs {
  CacheView C;
  SeqTables S;
  const bf16* x;
  bf16* out;
  float* lse;
  int64_t xs[3], os[3];
};

// The plainest form: one block per (row, head, sequence), its four warps take
// keys in turn with a running maximum and sum, a lane holds d / 32 dimensions.
// grid (n, heads, batch), block 128.
template <int D, bool I8>
__global__ void __launch_bounds__(128) k_cache_attend(AttendArgs A) {
  constexpr int DL = D / 32;
  __shared__ float so[4][D], sm[4], sl[4];
  const CacheView& C = A.C;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int len, nv;
  if (!seq_rows(A.S, C.P, b, &len, &nv) && threadIdx.x == 0) cache_error(C);
  const int64_t p = (int64_t)len + t;
  float q[DL], o[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) {
    q[i] = t < nv ? __bfloat162float(A.x[b * A.xs[0] + h * A.xs[1] + t * A.xs[2] + i * 32 + lane])
                  : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const float scale = 1.f / sqrtf((float)D);
  for (int64_t j = warp; t < nv && j <= p; j += 4) {
    const int id = page_of(C, A.S, b, (int)(j / C.P));
    if (id < 0) {
      if (lane == 0) cache_error(C);
      continue;
    }
    const int slot = (int)(j % C.P);
    const int64_t base = page_base(C, id, h), hs = (int64_t)id * C.H + h;
    float k[DL], v[DL], dot = 0.f;
#pragma unroll
    for (int i = 0; i < DL; ++i) {
      const int dim = i * 32 + lane;
      const int64_t ka = base + slot * D + dim;
      const int64_t va = base + slot / kGroup * kGroup * D + dim * kGroup + slot % kGroup;
      if constexpr (I8) {
        k[i] = static_cast<int8_t*>(C.k)[ka] * C.kscale[hs];
        v[i] = static_cast<int8_t*>(C.v)[va] * C.vscale[hs];
      } else {
        k[i] = __bfloat162float(static_cast<bf16*>(C.k)[ka]);
        v[i] = __bfloat162float(static_cast<bf16*>(C.v)[va]);
      }
      dot = fmaf(q[i], k[i], dot);
    }
    dot = warp_sum(dot) * C.kinv[hs * C.P + slot] * scale;
    if (j == p) dot = kSelfLogit;
    const float mn = fmaxf(m, dot), corr = expf(m - mn), e = expf(dot - mn);
    m = mn;
    l = l * corr + e;
#pragma unroll
    for (int i = 0; i < DL; ++i) o[i] = o[i] * corr + e * v[i];
  }
#pragma unroll
  for (int i = 0; i < DL; ++i) so[warp][i * 32 + lane] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < 4; ++w) ll += sl[w] != 0.f ? sl[w] * expf(sm[w] - mm) : 0.f;
  for (int dim = threadIdx.x; dim < D; dim += 128) {
    float s = 0.f;
    for (int w = 0; w < 4; ++w) s += sl[w] != 0.f ? so[w][dim] * expf(sm[w] - mm) : 0.f;
    A.out[b * A.os[0] + h * A.os[1] + t * A.os[2] + dim] =
        __float2bfloat16_rn(ll != 0.f ? s / ll : 0.f);
  }
  if (threadIdx.x == 0)
    A.lse[((int64_t)b * C.H + h) * A.S.n + t] = ll != 0.f ? mm + logf(ll) : -INFINITY;
}

}  // namespace lsh
