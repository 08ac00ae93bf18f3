// Rotary positions with one to four axes.
//
// Pair (lo, hi) turns by t = position of its axis * frequency:
//   lo' = lo cos t - hi sin t,   hi' = lo sin t + hi cos t.
// t reaches millions of turns, so it is formed and reduced to a fraction of a
// turn in fp64 (the product of an int32 and an fp32 is exact there up to 2^29);
// the sine and cosine of the fraction are fp32.
#pragma once

#include "common.cuh"
#include "lsh_attn.h"

namespace lsh {

// lsh_rope_axes with its prefix sums, by value to the kernels.
struct RotPlan {
  int axes, adjacent;
  int pairs;                            // rotated pairs, all axes
  int off[LSH_ROPE_MAX_AXES];           // first dimension of each axis
  int half[LSH_ROPE_MAX_AXES];          // pairs of each axis
};

// Axis of rotated pair p (pairs are numbered through the axes).
__device__ __forceinline__ int rot_axis(const RotPlan& r, int p) {
  int a = 0;
#pragma unroll
  for (int i = 1; i < LSH_ROPE_MAX_AXES; ++i)
    if (i < r.axes && 2 * p >= r.off[i]) a = i;
  return a;
}

// cos and sin of position * frequency.
__device__ __forceinline__ void rot_angle(int32_t pos, float freq, float* c, float* s) {
  double turns = (double)pos * (double)freq * 0.15915494309189533577;  // 1 / (2 pi)
  turns -= rint(turns);
  sincospif(2.0f * (float)turns, s, c);
}

// W consecutive elements of T, loaded and stored as one access, as fp32.
template <typename T, int W>
struct Pack {
  static constexpr int kBytes = W * (int)sizeof(T);
  static __device__ __forceinline__ void load(const T* p, float* f) {
    if constexpr (kBytes == 16) {
      Vec16<T>::unpack(*reinterpret_cast<const uint4*>(p), f);
    } else {
      alignas(16) T e[W];
      if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
      else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
      else e[0] = p[0];
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = Elem<T>::to_f(e[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
    alignas(16) T e[W];
#pragma unroll
    for (int i = 0; i < W; ++i) e[i] = Elem<T>::from_f(f[i]);
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(e);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<uint32_t*>(e);
    else p[0] = e[0];
  }
};

// Slot s of a row, s < d / (2 W): W pairs, held in two runs of W dimensions
// that start at *a and *b. Pairing by halves: the runs are the pairs' first and
// second dimensions (W divides every axis's pairs, so a run stays in its axis);
// adjacent: the runs follow one another and hold both. *first is the number of
// the first pair; pairs from r.pairs on are not rotated.
template <int W, bool ADJ>
__device__ __forceinline__ void rot_slot(const RotPlan& r, int s, int* a, int* b, int* first) {
  const int p = s * W;
  *first = p;
  if (ADJ || p >= r.pairs) {
    *a = 2 * p;
    *b = 2 * p + W;
  } else {
    const int ax = rot_axis(r, p);
    *a = r.off[ax] / 2 + p;  // off + (p - off / 2)
    *b = *a + r.half[ax];
  }
}

// The first `turned` of a slot's W pairs turned by (c, s) in place, the others
// left as they are (not multiplied: they may hold infinities): x of run a, y of
// run b.
template <int W, bool ADJ>
__device__ __forceinline__ void rot_apply(float (&x)[W], float (&y)[W], const float (&c)[W],
                                          const float (&s)[W], int turned) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i >= turned) continue;
    float lo, hi;
    if (ADJ && W > 1) {
      lo = 2 * i < W ? x[(2 * i) % W] : y[(2 * i) % W];
      hi = 2 * i + 1 < W ? x[(2 * i + 1) % W] : y[(2 * i + 1) % W];
    } else {
      lo = x[i];
      hi = y[i];
    }
    const float l2 = lo * c[i] - hi * s[i], h2 = lo * s[i] + hi * c[i];
    if (ADJ && W > 1) {
      (2 * i < W ? x[(2 * i) % W] : y[(2 * i) % W]) = l2;
      (2 * i + 1 < W ? x[(2 * i + 1) % W] : y[(2 * i + 1) % W]) = h2;
    } else {
      x[i] = l2;
      y[i] = h2;
    }
  }
}

constexpr int kRopeHeads = 4;  // heads loaded together by a thread

struct RopeArgs {
  const int32_t* pos;
  const float* freqs;
  int B, H, n, d;
  int heads_per;       // heads a thread turns with the same sines
  int head_groups;
  int64_t pos_axis, pos_batch;  // strides of positions
  int64_t xs[3], os[3];
  float sign;          // -1: the inverse rotation
  RotPlan rot;
};

// One thread holds a token's slot: its W sines and cosines serve every head of
// its group, so that the angles cost a fraction 1/heads_per of the rows.
// grid (blocks over tokens x slots, batch x head groups), block 256.
template <typename T, int W, bool ADJ>
__global__ void __launch_bounds__(256) k_rope(const T* x, T* out, RopeArgs A) {
  const int slots = A.d / (2 * W);
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t tok = id / slots;
  const int slot = (int)(id - tok * slots);
  if (tok >= A.n) return;
  for (int64_t bg = blockIdx.y; bg < (int64_t)A.B * A.head_groups; bg += gridDim.y) {
    const int b = (int)(bg / A.head_groups), h0 = (int)(bg % A.head_groups) * A.heads_per;
    const int h1 = min(h0 + A.heads_per, A.H);
    int ra, rb, p;
    rot_slot<W, ADJ>(A.rot, slot, &ra, &rb, &p);
    float c[W], s[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (p + i < A.rot.pairs) {
        const int ax = rot_axis(A.rot, p + i);
        rot_angle(A.pos[ax * A.pos_axis + b * A.pos_batch + tok], A.freqs[p + i], &c[i], &s[i]);
        s[i] *= A.sign;
      }
    }
    const int turned = A.rot.pairs - p;
    const T* xp = x + b * A.xs[0] + tok * A.xs[2];
    T* op = out + b * A.os[0] + tok * A.os[2];
    // heads in batches, all of a batch loaded before the first is stored: x and
    // out may be the same rows, so the compiler cannot do this by itself
    for (int h = h0; h < h1; h += kRopeHeads) {
      float u[kRopeHeads][W], w[kRopeHeads][W];
#pragma unroll
      for (int k = 0; k < kRopeHeads; ++k)
        if (h + k < h1) {
          Pack<T, W>::load(xp + (h + k) * A.xs[1] + ra, u[k]);
          Pack<T, W>::load(xp + (h + k) * A.xs[1] + rb, w[k]);
        }
#pragma unroll
      for (int k = 0; k < kRopeHeads; ++k)
        if (h + k < h1) {
          rot_apply<W, ADJ>(u[k], w[k], c, s, turned);
          Pack<T, W>::store(op + (h + k) * A.os[1] + ra, u[k]);
          Pack<T, W>::store(op + (h + k) * A.os[1] + rb, w[k]);
        }
    }
  }
}

}  // namespace lsh
