// Rotary positions with one to four axes.
//
// Pair (lo, hi) turns by t = position of its axis * frequency:
//   lo' = lo cos t - hi sin t,   hi' = lo sin t + hi cos t.
// t reaches millions of turns, of which only the fraction of a turn counts. A
// frequency is therefore held as a fraction of a turn in 64 bits of fixed point:
// a position times it, modulo 2^64, is the fraction, exact but for the position
// times 2^-65, in three integer operations (products in fp64, reduced there, took
// a third of the instructions of a kernel that has to keep up with DRAM).
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

// A frequency, radians a position, as a fraction of a turn in units of 2^-64.
// 1 / (2 pi) is taken to 107 bits, so that the product is good to 2^-64.
__device__ __forceinline__ uint2 rot_phase(float freq) {
  const double f = (double)freq, hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double p = f * hi, e = fma(f, hi, -p) + f * lo;
  // the fraction of p in [0, 1) has 53 bits; what is left of p is below 2^-53 of it
  const uint64_t u = (uint64_t)((p - floor(p)) * 0x1p64) + (uint64_t)(int64_t)(e * 0x1p64);
  return make_uint2((uint32_t)u, (uint32_t)(u >> 32));
}

// cos and sin of position * frequency. FAST: the sine and cosine units, off by
// 2^-21 at most: for results that are rounded to bf16.
template <bool FAST>
__device__ __forceinline__ void rot_angle(int32_t pos, uint2 phase, float* c, float* s) {
  // bits 32 .. 63 of pos * phase, pos being signed
  const uint32_t p = (uint32_t)pos;
  const int32_t turn =
      (int32_t)(__umulhi(p, phase.x) + p * phase.y - (pos < 0 ? phase.x : 0u));
  if constexpr (FAST) {
    __sincosf((float)turn * 1.46291807926715968e-9f, s, c);  // 2 pi / 2^32: [-pi, pi]
  } else {
    sincospif((float)turn * 0x1p-31f, s, c);
  }
}

// W consecutive elements of T (W = 1 too), loaded as one access, as fp32.
template <typename T, int W>
__device__ __forceinline__ void load_w(const T* p, float* f) {
  constexpr int kBytes = W * (int)sizeof(T);
  if constexpr (kBytes == 16) {
    Vec16<T>::unpack(*reinterpret_cast<const uint4*>(p), f);
  } else {
    alignas(8) T e[W];
    if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
    else e[0] = p[0];
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = Elem<T>::to_f(e[i]);
  }
}
// fp32 values rounded to T, 16 bytes.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f) {
  alignas(16) T e[16 / sizeof(T)];
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i) e[i] = Elem<T>::from_f(f[i]);
  return *reinterpret_cast<uint4*>(e);
}

// A thread turns a piece of N consecutive dimensions (16 bytes), so rows are read
// and written by whole sectors whatever the axes are. It needs the pairs' other
// dimensions too: neighbouring pairs lie inside the piece (ADJ); of halves the
// others lie in runs of W dimensions, which a lane of the same row holds. W
// divides every axis's pairs, so a run's partners are a run.
template <int N, int W, bool ADJ>
struct Piece {
  static constexpr int kRuns = ADJ ? 1 : N / W;
  static constexpr int kPairs = ADJ ? N / 2 : N;  // angles
  int other[kRuns];       // halves: first partner dimension of each run
  int pair[kRuns];        // first pair of each run
  uint32_t first, turned;  // bit per run: first half; bit per angle: is rotated

  __device__ __forceinline__ void place(const RotPlan& R, int dim0) {
    first = turned = 0;
    if constexpr (ADJ) {
      pair[0] = dim0 / 2;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) turned |= (uint32_t)(pair[0] + i < R.pairs) << i;
      if (!turned) pair[0] = 0;
    } else {
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        const int dim = dim0 + k * W;
        other[k] = dim;
        pair[k] = 0;
        if (dim >= 2 * R.pairs) continue;
        int a = 0;
#pragma unroll
        for (int i = 1; i < LSH_ROPE_MAX_AXES; ++i)
          if (i < R.axes && dim >= R.off[i]) a = i;
        const int at = dim - R.off[a], h = R.half[a];
        const bool lo = at < h;
        other[k] = lo ? dim + h : dim - h;
        pair[k] = R.off[a] / 2 + (lo ? at : at - h);
        first |= (uint32_t)lo << k;
        turned |= ((1u << W) - 1) << (k * W);
      }
    }
  }
  // pair of angle i, and the sign its sine takes
  __device__ __forceinline__ int pair_of(int i) const { return ADJ ? pair[0] + i : pair[i / W] + i % W; }
  __device__ __forceinline__ float sign_of(int i) const {
    return !ADJ && (first >> (i / W) & 1) ? -1.f : 1.f;
  }
  // x: the piece; y: its partners (halves); c, s: of every angle, s signed.
  // Spelled out, so that every kernel rounds alike; what is not turned is copied,
  // not multiplied: it may be infinite.
  __device__ __forceinline__ void turn(float (&x)[N], const float (&y)[N], const float (&c)[kPairs],
                                       const float (&s)[kPairs]) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if (!(turned >> i & 1)) continue;
      if constexpr (ADJ) {
        const float lo = x[2 * i], hi = x[2 * i + 1];
        x[2 * i] = __fmaf_rn(lo, c[i], __fmul_rn(hi, -s[i]));
        x[2 * i + 1] = __fmaf_rn(hi, c[i], __fmul_rn(lo, s[i]));
      } else {
        x[i] = __fmaf_rn(x[i], c[i], __fmul_rn(y[i], s[i]));
      }
    }
  }
};

constexpr int kRopeHeads = 4;  // heads loaded together by a thread

struct RopeArgs {
  const int32_t* pos;
  const float* freqs;
  int B, H, n;
  int heads_per;       // heads a thread turns with the same sines
  int head_groups;
  int64_t pos_axis, pos_batch;  // strides of positions
  int64_t xs[3], os[3];
  float sign;          // -1: the inverse rotation
  RotPlan rot;
};

// One thread holds a piece of a token: its sines and cosines serve every head of
// its group, so that the angles cost a fraction 1 / heads_per of the rows. Bound
// by DRAM: what counts is whole sectors and bytes in flight, four heads' pieces
// a thread. Halves: the lanes of a row form each angle once and share them, and
// pass one another their pieces, through shared memory (partners read from
// global memory as well: 95 us instead of __ROPE_IMAGE__ us at B8 H8 n12288 d64 with axes
// 24, 24, 16).
// grid (blocks over tokens x pieces, batch x head groups), block 256.
template <typename T, int D, int W, bool ADJ>
__global__ void __launch_bounds__(256) k_rope(const T* x, T* out, RopeArgs A) {
  constexpr int N = 16 / sizeof(T), kPieces = D / N;  // a row's pieces lie in one warp
  constexpr int kTok = 256 / kPieces;
  using P = Piece<N, W, ADJ>;
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ float ct[ADJ ? 1 : kTok * D / 2], st[ADJ ? 1 : kTok * D / 2];
  __shared__ uint2 phase[D / 2];
  __shared__ uint8_t axis[D / 2];
  __shared__ uint4 swap[ADJ ? 1 : kRopeHeads][256];
  const int64_t tok0 = (int64_t)blockIdx.x * kTok;
  const int tl = threadIdx.x / kPieces, dim0 = threadIdx.x % kPieces * N;
  const int64_t tok = tok0 + tl;
  const bool in = tok < A.n;
  const int pairs = A.rot.pairs;
  if (threadIdx.x < pairs) {
    phase[threadIdx.x] = rot_phase(A.freqs[threadIdx.x]);
    axis[threadIdx.x] = (uint8_t)rot_axis(A.rot, threadIdx.x);
  }
  __syncthreads();
  P piece;
  piece.place(A.rot, dim0);
  for (int64_t bg = blockIdx.y; bg < (int64_t)A.B * A.head_groups; bg += gridDim.y) {
    const int b = (int)(bg / A.head_groups), h0 = (int)(bg % A.head_groups) * A.heads_per;
    const int h1 = min(h0 + A.heads_per, A.H);
    const T* xp = x + b * A.xs[0] + (in ? tok : 0) * A.xs[2] + dim0;
    T* op = out + b * A.os[0] + tok * A.os[2] + dim0;
    const int32_t* pos = A.pos + b * A.pos_batch;
    float c[P::kPairs], s[P::kPairs];
    if constexpr (!ADJ) {
      __syncthreads();  // the angles of the batch before have been taken
      const int toks = (int)min((int64_t)kTok, A.n - tok0);
      for (int i = threadIdx.x; i < toks * pairs; i += 256) {
        const int p = i % pairs;
        rot_angle<kFast>(pos[axis[p] * A.pos_axis + tok0 + i / pairs], phase[p], &ct[i], &st[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < P::kPairs; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (in && (piece.turned >> i & 1)) {
        const int p = piece.pair_of(i);
        if constexpr (ADJ) {
          rot_angle<kFast>(pos[axis[p] * A.pos_axis + tok], phase[p], &c[i], &s[i]);
        } else {
          c[i] = ct[tl * pairs + p];
          s[i] = st[tl * pairs + p];
        }
        s[i] *= A.sign * piece.sign_of(i);
      }
    }
    // heads in batches, all of a batch loaded before the first is stored (x and
    // out may be the same rows)
    for (int h = h0; h < h1; h += kRopeHeads) {
      uint4 u[kRopeHeads];
#pragma unroll
      for (int k = 0; k < kRopeHeads; ++k)
        if (h + k < h1) u[k] = *reinterpret_cast<const uint4*>(xp + (h + k) * A.xs[1]);
      if constexpr (!ADJ) {
#pragma unroll
        for (int k = 0; k < kRopeHeads; ++k) swap[k][threadIdx.x] = u[k];
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < kRopeHeads; ++k)
        if (h + k < h1 && in) {
          float f[N], y[N];
          Vec16<T>::unpack(u[k], f);
          if constexpr (!ADJ) {
            const T* row = reinterpret_cast<const T*>(&swap[k][tl * kPieces]);
#pragma unroll
            for (int r = 0; r < P::kRuns; ++r) load_w<T, W>(row + piece.other[r], &y[r * W]);
          }
          piece.turn(f, y, c, s);
          *reinterpret_cast<uint4*>(op + (h + k) * A.os[1]) = pack16<T>(f);
        }
      if constexpr (!ADJ) __syncwarp();
    }
  }
}

}  // namespace lsh
