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
#include "sm100.cuh"

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
// 1 / (2 pi) is taken to 107 bits, so that the product is good to 2^-63 for frequencies
// up to 2^45. That of a negative one is the negative of its opposite's: its own
// distance from the next lower turn would keep 53 bits.
__device__ __forceinline__ uint2 rot_phase(float freq) {
  const double f = fabs((double)freq), hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double p = f * hi, e = fma(f, hi, -p) + f * lo;
  // the fraction of p in [0, 1) has 53 bits; what is left of p is below 2^-53 of it
  uint64_t u = (uint64_t)((p - floor(p)) * 0x1p64) + (uint64_t)(int64_t)(e * 0x1p64);
  if (freq < 0.f) u = 0 - u;
  return make_uint2((uint32_t)u, (uint32_t)(u >> 32));
}

// cos and sin of position * frequency. FAST: the sine and cosine units, off by
// 2^-21 at most: for results that are rounded to bf16. Else of the angle's leading
// 24 bits, which fp32 holds exactly, and turned on by the rest, d < 2^-22 (its square is
// nothing): the angle rounded to fp32 would be off by 2^-23, more than a sine's own step
// (8 heads of fp32: no difference; one head of 131072 rows: 67.7 us instead of 65.6).
template <bool FAST>
__device__ __forceinline__ void rot_angle(int32_t pos, uint2 phase, float* c, float* s) {
  // bits 32 .. 63 of pos * phase, pos being signed
  const uint32_t p = (uint32_t)pos;
  const int32_t turn =
      (int32_t)(__umulhi(p, phase.x) + p * phase.y - (pos < 0 ? phase.x : 0u));
  if constexpr (FAST) {
    __sincosf((float)turn * 1.46291807926715968e-9f, s, c);  // 2 pi / 2^32: [-pi, pi]
  } else {
    sincospif((float)(turn & ~127) * 0x1p-31f, s, c);
    const float d = (__uint_as_float(0x4b000000u | (turn & 127)) - 8388608.f) * 1.46291807926715968e-9f;
    const float s0 = *s;
    *s = fmaf(*c, d, s0);
    *c = fmaf(-s0, d, *c);
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
  static constexpr uint32_t kAll = (1u << kPairs) - 1;
  int other[kRuns];       // halves: first partner dimension of each run
  int pair[kRuns];        // first pair of each run
  uint32_t first, turned;  // bit per run: first half; bit per angle: is rotated

  // Runs that are not rotated find zeros as partners, at `zeros` from the row.
  __device__ __forceinline__ void place(const RotPlan& R, int dim0, int zeros) {
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
        other[k] = zeros;
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
  // Spelled out, so that every kernel rounds alike. What is not turned is copied:
  // halves with c = 1, s = -0 and zeros as partners (x + -0 is x, of any x);
  // neighbours by leaving them out (a partner may be infinite).
  __device__ __forceinline__ void turn(float (&x)[N], const float (&y)[N], const float (&c)[kPairs],
                                       const float (&s)[kPairs]) const {
    if constexpr (!ADJ) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = __fmaf_rn(x[i], c[i], __fmul_rn(y[i], s[i]));
    } else if (turned == kAll) {
      pairs<true>(x, c, s);
    } else {
      pairs<false>(x, c, s);
    }
  }
  template <bool ALL>
  __device__ __forceinline__ void pairs(float (&x)[N], const float (&c)[kPairs],
                                        const float (&s)[kPairs]) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (!ALL && !(turned >> i & 1)) continue;
      const float lo = x[2 * i], hi = x[2 * i + 1];
      x[2 * i] = __fmaf_rn(lo, c[i], __fmul_rn(hi, -s[i]));
      x[2 * i + 1] = __fmaf_rn(hi, c[i], __fmul_rn(lo, s[i]));
    }
  }
};

constexpr int kRopeHeads = 4;  // heads of a batch

struct RopeArgs {
  const int32_t* pos;
  const float* freqs;
  int B, H, n;
  int tiles;           // of a sequence's tokens
  int heads_per;       // heads a thread turns with the same sines
  int head_groups;
  int step_tile, step_group, step_b;  // gridDim.x jobs
  int64_t pos_axis, pos_batch;  // strides of positions
  int64_t xs[3], os[3];
  float sign;          // -1: the inverse rotation
  RotPlan rot;
};

// A job is a tile of tokens (256 pieces of rows) for a group of heads; a block
// takes one or more in turn. A thread's sines and cosines serve every head of the
// group: the angles cost a fraction 1 / heads_per of the rows. What bounds the
// kernel besides DRAM is the instructions beside the rotation itself: where a
// piece lies, the phases, the angles. Rows come by cp.async, two batches of heads
// ahead, and are under way meanwhile. Halves: the lanes of a row form each angle
// once and find their partners' pieces in shared memory. Measured: 45.8 us at B1 H8
// n65536 d128, neighbours (0.89 of the copy rate), 41 us at B8 H8 n12288 d64, axes
// 24, 24, 16 by halves (0.75; with partners read from global memory too, 95 us; a
// position fetched for each angle when it is formed, 43 us). Halves in runs of one or
// two take 76 to 115 registers: two or three blocks an SM (axes 44, 42, 42 at the first of
// these sizes 61.6 us, 0.67; axes 10, 14 at the second 53.9, 0.57).
// grid (blocks), block 256.
template <typename T, int D, int W, bool ADJ>
__global__ void __launch_bounds__(256, ADJ || W < 4 ? 0 : 5) k_rope(const T* x, T* out, RopeArgs A) {
  constexpr int N = 16 / sizeof(T), kPieces = D / N;  // a row's pieces lie in one warp
  constexpr int kTok = 256 / kPieces;
  constexpr bool kFast = sizeof(T) == 2;
  using P = Piece<N, W, ADJ>;
  __shared__ float ct[ADJ ? 1 : kTok * D / 2], st[ADJ ? 1 : kTok * D / 2];
  __shared__ uint4 rows[2][kRopeHeads][257];  // a batch of heads each; the last piece: zeros
  __shared__ uint2 phase[D / 2];
  __shared__ uint8_t axis[D / 2];
  __shared__ int32_t pos[LSH_ROPE_MAX_AXES * kTok];
  const int tl = threadIdx.x / kPieces, dim0 = threadIdx.x % kPieces * N;
  const int pairs = A.rot.pairs;
  const int batches = (A.heads_per + kRopeHeads - 1) / kRopeHeads;

  // jobs are numbered through tiles, head groups and sequences
  struct Job {
    int tile, group, b;
  };
  auto job_of = [&](uint32_t i) {
    const uint32_t rest = i / (uint32_t)A.tiles;
    return Job{(int)(i - rest * A.tiles), (int)(rest % (uint32_t)A.head_groups),
               (int)(rest / (uint32_t)A.head_groups)};
  };
  auto next = [&](Job& j) {  // the job gridDim.x on: digit by digit
    j.tile += A.step_tile;
    j.group += A.step_group;
    j.b += A.step_b;
    if (j.tile >= A.tiles) {
      j.tile -= A.tiles;
      ++j.group;
    }
    if (j.group >= A.head_groups) {
      j.group -= A.head_groups;
      ++j.b;
    }
  };
  // batches of heads, numbered through the block's jobs, two under way
  Job ahead = job_of(blockIdx.x);
  Job job = ahead;
  int batch_f = 0, buf = 0;
  auto fetch = [&](int to) {
    if (ahead.b < A.B) {
      const int h = ahead.group * A.heads_per + batch_f * kRopeHeads;
      const int n = min((ahead.group + 1) * A.heads_per, A.H) - h;
      const int64_t tok = (int64_t)ahead.tile * kTok + tl;
      const T* xp = x + ahead.b * A.xs[0] + h * A.xs[1] + tok * A.xs[2] + dim0;
      if (tok < A.n) {
#pragma unroll
        for (int k = 0; k < kRopeHeads; ++k, xp += A.xs[1])
          if (k < n) sm100::cp_async16_zfill(&rows[to][k][threadIdx.x], xp, true);
      }
      if (++batch_f == batches) {
        batch_f = 0;
        next(ahead);
      }
    }
    sm100::cp_async_commit();
  };
  fetch(0);
  fetch(1);
  if (threadIdx.x < pairs) {
    phase[threadIdx.x] = rot_phase(A.freqs[threadIdx.x]);
    axis[threadIdx.x] = (uint8_t)rot_axis(A.rot, threadIdx.x);
  }
  if (!ADJ && threadIdx.x < 2 * kRopeHeads)
    rows[threadIdx.x / kRopeHeads][threadIdx.x % kRopeHeads][256] = make_uint4(0, 0, 0, 0);
  P piece;
  piece.place(A.rot, dim0, (256 - tl * kPieces) * N);
  // a thread's first angle of a tile's, and its stride: no division in the loop
  const int first_tok = threadIdx.x / pairs, first_pair = threadIdx.x % pairs;
  const int step_tok = 256 / pairs, step_pair = 256 % pairs;
  // a job's positions, fetched while the one before it is worked on
  int32_t ahead_pos = 0;
  auto fetch_pos = [&](const Job& j) {
    const int a = threadIdx.x / kTok, t = threadIdx.x % kTok;
    const int64_t tok = (int64_t)j.tile * kTok + t;
    if (j.b < A.B && a < A.rot.axes && tok < A.n)
      ahead_pos = A.pos[a * A.pos_axis + j.b * A.pos_batch + tok];
  };
  fetch_pos(job);
  float sign[P::kPairs];
#pragma unroll
  for (int i = 0; i < P::kPairs; ++i) sign[i] = A.sign * piece.sign_of(i);

  while (job.b < A.B) {
    const int h0 = job.group * A.heads_per, h1 = min(h0 + A.heads_per, A.H);
    const int64_t tok0 = (int64_t)job.tile * kTok;
    const bool in = tok0 + tl < A.n;
    T* oh = out + job.b * A.os[0] + h0 * A.os[1] + (tok0 + tl) * A.os[2] + dim0;
    float c[P::kPairs], s[P::kPairs];
    // (the angles of the job before have been taken: the barrier behind them)
    if (threadIdx.x < LSH_ROPE_MAX_AXES * kTok) pos[threadIdx.x] = ahead_pos;
    __syncthreads();
    Job after = job;
    next(after);
    fetch_pos(after);
    if constexpr (!ADJ) {
      const int toks = (int)min((int64_t)kTok, A.n - tok0);
      for (int t = first_tok, p = first_pair; t < toks;) {
        rot_angle<kFast>(pos[axis[p] * kTok + t], phase[p], &ct[t * pairs + p],
                         &st[t * pairs + p]);
        t += step_tok;
        p += step_pair;
        if (p >= pairs) {
          p -= pairs;
          ++t;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < P::kPairs; ++i) {
      c[i] = 1.f;
      s[i] = -0.f;
      if (in && (piece.turned >> i & 1)) {
        const int p = piece.pair_of(i);
        if constexpr (ADJ) {
          rot_angle<kFast>(pos[axis[p] * kTok + tl], phase[p], &c[i], &s[i]);
        } else {
          c[i] = ct[tl * pairs + p];
          s[i] = st[tl * pairs + p];
        }
        s[i] *= sign[i];
      }
    }
    __syncthreads();  // positions and angles have been taken
    job = after;
    for (int h = h0; h < h0 + batches * kRopeHeads; h += kRopeHeads) {
      sm100::cp_async_wait_prev();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kRopeHeads; ++k, oh += A.os[1])
        if (h + k < h1) {
          const uint4* row = &rows[buf][k][tl * kPieces];
          float f[N], y[N];
          Vec16<T>::unpack(rows[buf][k][threadIdx.x], f);
          if constexpr (!ADJ) {
#pragma unroll
            for (int r = 0; r < P::kRuns; ++r)
              load_w<T, W>(reinterpret_cast<const T*>(row) + piece.other[r], &y[r * W]);
          }
          piece.turn(f, y, c, s);
          if (in) *reinterpret_cast<uint4*>(oh) = pack16<T>(f);
        }
      __syncwarp();
      fetch(buf);
      buf ^= 1;
    }
  }
}

}  // namespace lsh
