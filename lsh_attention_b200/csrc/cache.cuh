// The paged cache: what its kernels share, and the kernels that write rows into
// it and read them back.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "lsh_attn.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace lsh {

using bf16 = __nv_bfloat16;
constexpr int kGroup = 16;  // tokens of a v group: no group crosses a page

struct CacheView {
  void* k;
  void* v;
  float* kinv;
  float* kscale;
  float* vscale;
  WsHeader* status;  // NULL: errors are not recorded
  int pages, H, P, d;
};

struct SeqTables {
  const int32_t* table;
  const int32_t* len;
  const int32_t* valid;  // NULL: n
  int B, n, max_pages;
};

__device__ __forceinline__ void cache_error(const CacheView& C) {
  if (C.status) record_status(C.status, 6u /* LSH_ERR_DEVICE */);
}

// Sequence b: its tokens before the call's rows, and how many rows it has; a
// sequence whose numbers are out of range has none. False if they were.
__device__ __forceinline__ bool seq_rows(const SeqTables& S, int P, int b, int* len, int* nv) {
  const int l = S.len[b], v = S.valid ? S.valid[b] : S.n;
  const bool ok = l >= 0 && v >= 0 && v <= S.n && (int64_t)l + v <= (int64_t)S.max_pages * P;
  *len = ok ? l : 0;
  *nv = ok ? v : 0;
  return ok;
}

// Page of sequence b's tokens page * P ..; -1 if the table's number is bad.
// `page` is below max_pages.
__device__ __forceinline__ int page_of(const CacheView& C, const SeqTables& S, int b, int page) {
  const int id = S.table[(int64_t)b * S.max_pages + page];
  return id >= 0 && id < C.pages ? id : -1;
}

// First element of (page, head) in k or v.
__device__ __forceinline__ int64_t page_base(const CacheView& C, int id, int h) {
  return ((int64_t)id * C.H + h) * C.P * C.d;
}

// Smallest power of two s >= 2^-126 with amax <= 127 s. amax finite, >= 0: with
// amax = f 2^e, f in [1, 2), that is 2^(e - 6), or 2^(e - 5) where f > 127 / 64.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 6 + ((b & 0x7fffffu) > 0x7e0000u);  // biased
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// 1 / s of a power of two s in [2^-126, 2^126].
__device__ __forceinline__ float recip2(float s) {
  return __uint_as_float(0x7f000000u - __float_as_uint(s));
}

// x / s rounded to the nearest integer (ties to even), in the low byte. rs = 1 / s
// is a power of two, so the product is exact; 1.5 2^23 added in the same
// instruction rounds it and leaves it in the mantissa. `odd`: x may be infinite or
// NaN: kept in [-127, 127], NaN to 0 (finite ones are, by the choice of s).
__device__ __forceinline__ uint32_t quant(float x, float rs, bool odd) {
  if (odd) x = x == x ? fminf(fmaxf(x, -127.f * recip2(rs)), 127.f * recip2(rs)) : 0.f;
  return __float_as_uint(fmaf(x, rs, 12582912.f));
}
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float rs, bool odd) {
  return __byte_perm(__byte_perm(quant(a, rs, odd), quant(b, rs, odd), 0x0040),
                     __byte_perm(quant(c, rs, odd), quant(d, rs, odd), 0x0040), 0x5410);
}

// Four int8 times s, a power of two, as bf16 (exact): each byte is put into the
// mantissa of 2^23, as q + 128, and 2^23 + 128 taken off.
__device__ __forceinline__ uint2 i8_values(uint32_t w, float s) {
  w ^= 0x80808080u;
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + i)) - 8388736.f) * s;
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Four 8x8 tiles of 16-bit values, transposed: lane (g = lane / 4, t = lane % 4)
// gets the elements [2t][g] and [2t + 1][g] of each; lanes 8 i .. 8 i + 7 give
// the addresses of the rows of tile i.
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], const void* row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(row)));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

struct AppendArgs {
  CacheView C;
  SeqTables S;
  RotPlan rot;  // axes 0: no rotation
  const bf16* x;
  const bf16* v;
  const int32_t* pos;
  const float* freqs;
  bf16* xr;  // may be NULL
  int64_t pos_axis, pos_batch;
  int64_t xs[3], vs[3], os[3];
  int heads_per;  // heads a block takes one after the other
};

// How the rows are turned.
enum { kTurnNone = 0, kTurnAdjacent = 1, kTurnRuns = 2, kTurnSingles = 3 };

// Rows that a block has room for. bf16 tokens do not depend on one another: blocks
// of 32, aligned in the sequence. int8 ones share their page's scale, so a block
// has whole pages, 32 or more tokens; of larger pages into which a call can put no
// more than 17 rows, it has 32 rows from the group of the first new one on.
__host__ __device__ constexpr int append_rows(bool i8, int page, int n) {
  return !i8 || page < 32 || n <= 17 ? 32 : page;
}
// Angles of a row in shared memory, rounded up to whole float4.
__host__ __device__ constexpr int append_pairs(int pairs) { return (pairs + 3) / 4 * 4; }
constexpr size_t append_smem(int rows, int d, int pairs, int buffers) {
  return (size_t)rows * (buffers * 2 * (d * 2 + 16) + append_pairs(pairs) * 8) + 32 + 128;
}

// Tiles of two heads, and four blocks an SM; 128 rows of 128 leave room for one
// head and one block, which has more threads.
constexpr int append_buffers(int d, int rows) { return d * rows > 128 * 64 ? 1 : 2; }
constexpr int append_threads(int d, int rows) {
  return d * rows > 128 * 64 ? 1024 : d * rows > 64 * 64 ? 512 : 256;
}

// 1/||x|| of a row whose kLanes lanes hold its values by eight; of a row that is
// not there (not `in`), anything.
template <int kLanes>
__device__ __forceinline__ float inv_norm(const float (&f)[8], bool in) {
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
  const bool plain = !in || (ss > 0x1p-80f && ss < 0x1p100f);  // no square was lost
  if (__all_sync(~0u, plain)) return rsqrtf(ss);
  // scaled by a power of two near the row's largest value
  float m = 0.f;
  ss = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const int e = max(-126, min(126, (int)(__float_as_uint(m) >> 23) - 127));
  const float up = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int k = 0; k < 8; ++k) ss = fmaf(f[k] * up, f[k] * up, ss);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
  const float norm = sqrtf(ss) * __uint_as_float((uint32_t)(127 + e) << 23);
  return norm < 0x1p-126f ? 0.f : 1.f / norm;
}

// One block: R consecutive token slots of one sequence for a few heads. The sines
// of its tokens are formed once and serve its heads; the next two heads' rows
// travel (cp.async) meanwhile. A thread takes 16-byte pieces of rows of x: 1/||x||,
// the rotation with the partners from shared memory, the rotated piece out. v
// leaves through transposed 8x8 tiles (ldmatrix), so that a thread stores four
// tokens of a dimension together and a warp whole sectors of the groups. int8:
// pieces wait in registers for the page's largest magnitude (maxima of
// non-negative floats by integer atomicMax in shared memory: the same whatever the
// order); this block alone owns the page's head, so earlier rows are rounded again
// in place. A stream of rows in and out, bound by DRAM in bf16: 64
// us for 4 x 8192 rows of 8 heads of 128 with a rotation (0.80 of the copy rate; 48 us
// without one, which writes a third less). int8 is near none of
// its limits: two thirds of the issue slots, 41% of the warps active, waits at its four
// barriers a head among the first stalls, DRAM mostly idle: 95 us there (0.43); with every
// thread forming the scales itself, two of the barriers left out, 96.
// grid (blocks of rows, head groups, batch), block append_threads(D, R).
template <int D, bool I8, int R, int TURN>
__global__ void __launch_bounds__(append_threads(D, R), 1024 / append_threads(D, R))
    k_cache_append(AppendArgs A) {
  constexpr int kStride = D + 8;  // elements of a shared row: 16 bytes of padding
  constexpr int kPieces = D / 8;  // 16-byte pieces of a row
  constexpr int kThreads = append_threads(D, R), kWarps = kThreads / 32;
  constexpr int kPass = R * kPieces / kThreads;
  constexpr int kBuf = append_buffers(D, R);
  constexpr int W = TURN == kTurnSingles ? 1 : 4;
  constexpr bool ADJ = TURN == kTurnAdjacent;
  using P8 = Piece<8, W, ADJ>;
  const CacheView& C = A.C;
  const int b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = A.S.n;
  const int h0 = blockIdx.y * A.heads_per, h1 = min(h0 + A.heads_per, C.H);
  int len, nv;
  if (!seq_rows(A.S, C.P, b, &len, &nv) && blockIdx.x == 0 && tid == 0) cache_error(C);

  // rows of xr past the sequence's own: zeros
  if (A.xr) {
    const int t0 = max(nv, (int)min((int64_t)T, (int64_t)blockIdx.x * R));
    const int t1 = (int)min((int64_t)T, (int64_t)(blockIdx.x + 1) * R);
    const int pad = max(t1 - t0, 0) * (h1 - h0) * kPieces;
    for (int i = tid; i < pad; i += kThreads) {
      const int piece = i % kPieces, rest = i / kPieces;
      const int h = h0 + rest % (h1 - h0), t = t0 + rest / (h1 - h0);
      *reinterpret_cast<uint4*>(A.xr + b * A.os[0] + h * A.os[1] + t * A.os[2] + piece * 8) =
          make_uint4(0, 0, 0, 0);
    }
  }

  // the block's slots: positions base .. base + R - 1; new rows [r0, r1) of them
  const int span = I8 && C.P > R ? C.P : R;  // tokens between blocks
  int64_t base = (int64_t)(len / span + blockIdx.x) * span;
  const int64_t end = min(base + span, (int64_t)len + nv);
  if (span > R) base += max((int64_t)0, len - base) & ~(kGroup - 1);
  const int r0 = (int)max((int64_t)0, len - base);
  const int r1 = (int)max((int64_t)0, min((int64_t)R, end - base));
  if (r0 >= r1) return;
  const int tok0 = (int)(base - len);  // row r is the call's row tok0 + r

  extern __shared__ __align__(16) unsigned char smem[];
  bf16* tiles = reinterpret_cast<bf16*>(smem);  // [buffers][x, v][R][kStride]
  float* ct = reinterpret_cast<float*>(tiles + kBuf * 2 * R * kStride);
  const int pstride = append_pairs(A.rot.pairs);
  float* st = ct + R * pstride + 4;  // behind each the angle of what is not turned
  // int8: of at most two pages, largest magnitudes of x and v
  int* amax = reinterpret_cast<int*>(st + R * pstride + 4);
  __shared__ int ids[8];  // pages of the block's tokens
  __shared__ float scales[2][4];  // of a page: x old, new, v old, new
  __shared__ uint2 phase[D / 2];
  __shared__ uint8_t axis[D / 2];
  __shared__ int32_t pos[LSH_ROPE_MAX_AXES * R];

  // a thread's pieces are the same dimensions of rows kStep apart
  constexpr int kStep = kThreads / kPieces;
  const int dim0 = tid % kPieces * 8, row0 = tid / kPieces;
  auto fetch = [&](int h) {
    bf16* xt = tiles + ((h - h0) % kBuf) * 2 * R * kStride + row0 * kStride + dim0;
    const bf16* xg = A.x + b * A.xs[0] + h * A.xs[1] + (int64_t)(tok0 + row0) * A.xs[2] + dim0;
    const bf16* vg = A.v + b * A.vs[0] + h * A.vs[1] + (int64_t)(tok0 + row0) * A.vs[2] + dim0;
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      const int r = row0 + k * kStep;
      if (r >= r0 && r < r1) {
        sm100::cp_async16_zfill(xt + k * kStep * kStride, xg + k * kStep * A.xs[2], true);
        sm100::cp_async16_zfill(xt + (R + k * kStep) * kStride, vg + k * kStep * A.vs[2], true);
      }
    }
    sm100::cp_async_commit();
  };
  fetch(h0);
  if (kBuf == 2 && h0 + 1 < h1) fetch(h0 + 1);
  const int pages = (R + C.P - 1) / C.P;  // a block's rows lie in this many
  if (tid < pages) {
    // the page of the block's tokens from row tid * P on, if it has new ones
    int id = -1;
    if (tid * C.P < r1 && (tid + 1) * C.P > r0) {
      id = page_of(C, A.S, b, (int)((base + tid * C.P) / C.P));
      if (id < 0 && blockIdx.y == 0) cache_error(C);
    }
    ids[tid] = id;
  }
  P8 piece;
  int arow[P8::kRuns], afrom[P8::kRuns];  // a run's angles: afrom + arow * row
  if constexpr (TURN != kTurnNone) {
    const int pairs = A.rot.pairs;
    if (tid < 4) {
      ct[R * pstride + tid] = 1.f;
      st[R * pstride + tid] = -0.f;
    }
    // the padding of rows of x: zeros, the partners of what is not turned
    for (int r = tid; r < kBuf * R; r += kThreads)
      *reinterpret_cast<uint4*>(tiles + ((r / R) * 2 * R + r % R) * kStride + D) = make_uint4(0, 0, 0, 0);
    // every position at once: a load for each angle would wait in turn
    for (int i = tid; i < A.rot.axes * R; i += kThreads) {
      const int r = i % R;
      if (r >= r0 && r < r1) pos[i] = A.pos[(i / R) * A.pos_axis + b * A.pos_batch + tok0 + r];
    }
    if (tid < pairs) {
      phase[tid] = rot_phase(A.freqs[tid]);
      axis[tid] = (uint8_t)rot_axis(A.rot, tid);
    }
    __syncthreads();
    // rows go round a warp at a time: lanes take neighbouring pairs
    for (int r = r0 + warp; r < r1; r += kWarps)
      for (int p = lane; p < pairs; p += 32)
        rot_angle<true>(pos[axis[p] * R + r], phase[p], &ct[r * pstride + p], &st[r * pstride + p]);
    piece.place(A.rot, dim0, D);
#pragma unroll
    for (int q = 0; q < P8::kRuns; ++q) {
      const bool turned = piece.turned >> (q * W) & 1;
      arow[q] = turned ? pstride : 0;
      afrom[q] = turned ? piece.pair[q] : R * pstride;
    }
  }
  const int pmask = C.P - 1, pshift = __ffs(C.P) - 1;
  const int off0 = (int)base & pmask;  // row 0's slot: not 0 in a larger page only
  const int pf = r0 >> pshift, old = (off0 + r0) & pmask;  // the page of row r0, and its earlier rows

  for (int h = h0; h < h1; ++h) {
    if (kBuf == 2 && h + 1 < h1) sm100::cp_async_wait_prev();
    else sm100::cp_async_wait_all();
    if (I8 && tid < 4) amax[tid] = 0;
    __syncthreads();
    const bf16* xt = tiles + ((h - h0) % kBuf) * 2 * R * kStride;
    const bf16* vt = xt + R * kStride;
    bf16* xo = A.xr ? A.xr + b * A.os[0] + h * A.os[1] + (int64_t)(tok0 + row0) * A.os[2] + dim0 : nullptr;

    bool odd = false;  // int8: some value is not finite
    uint4 kept[I8 ? kPass : 1];
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      const int r = row0 + k * kStep;
      const bool in = r >= r0 && r < r1;
      if (!__any_sync(~0u, in)) continue;
      const bf16* row = xt + r * kStride;
      float f[8];
      uint4 u = *reinterpret_cast<const uint4*>(row + dim0);
      Vec16<bf16>::unpack(u, f);
      const float inv = inv_norm<kPieces>(f, in);
      const int pg = r >> pshift, id = ids[pg];
      // the row's slot in its page (page_base of id: [P][D] a head)
      const int64_t at = ((int64_t)id * C.H + h) * C.P + ((off0 + r) & pmask);
      // int8 stores NaN as 0: the row's logits are 0 then, as an infinite row's are
      if (in && id >= 0 && dim0 == 0) C.kinv[at] = I8 && inv != inv ? 0.f : inv;
      if constexpr (TURN != kTurnNone) {
        float y[8], c[P8::kPairs], s[P8::kPairs];
        if constexpr (ADJ) {
          load_w<float, 4>(ct + r * pstride + piece.pair[0], c);
          load_w<float, 4>(st + r * pstride + piece.pair[0], s);
        } else {
#pragma unroll
          for (int q = 0; q < P8::kRuns; ++q) {
            load_w<bf16, W>(row + piece.other[q], &y[q * W]);
            load_w<float, W>(ct + afrom[q] + r * arow[q], &c[q * W]);
            load_w<float, W>(st + afrom[q] + r * arow[q], &s[q * W]);
#pragma unroll
            for (int e = 0; e < W; ++e) s[q * W + e] *= piece.sign_of(q * W + e);
          }
        }
        piece.turn(f, y, c, s);
        u = pack16<bf16>(f);
      }
      if (in && xo) *reinterpret_cast<uint4*>(xo + k * kStep * A.os[2]) = u;
      if constexpr (I8) {
        kept[k] = u;
        // largest magnitudes, as bits with the sign taken off: finite ones compare
        // like integers; infinities and NaN are above 0x7f7f and left out
        uint32_t km = 0, vm = 0;
        const uint4 w = *reinterpret_cast<const uint4*>(vt + r * kStride + dim0);
        const uint32_t ku[4] = {u.x, u.y, u.z, u.w}, vu[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          km = __vmaxu2(km, ku[e] & 0x7fff7fffu);
          vm = __vmaxu2(vm, vu[e] & 0x7fff7fffu);
        }
        km = max(km & 0xffffu, km >> 16);
        vm = max(vm & 0xffffu, vm >> 16);
        if (in && max(km, vm) > 0x7f7fu) {
          odd = true;
          cache_error(C);
          km = vm = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t a = ku[e >> 1] >> (16 * (e & 1)) & 0x7fffu, c = vu[e >> 1] >> (16 * (e & 1)) & 0x7fffu;
            if (a <= 0x7f7fu) km = max(km, a);
            if (c <= 0x7f7fu) vm = max(vm, c);
          }
        }
        if (!in) km = vm = 0;
        // a warp's rows of a pass lie in one page of 16 at least
        km = __reduce_max_sync(~0u, km);
        vm = __reduce_max_sync(~0u, vm);
        if (lane == 0) {
          atomicMax(&amax[2 * pg], (int)(km << 16));
          atomicMax(&amax[2 * pg + 1], (int)(vm << 16));
        }
      } else if (in && id >= 0) {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(C.k) + at * D + dim0) = u;
      }
    }

    bool again = false;  // int8: values of the page's earlier rows are rounded again
    if constexpr (I8) {
      odd = __syncthreads_or(odd);
      if (tid < 2 * pages) {
        const int pg = tid >> 1, id = ids[pg];
        float was = 0.f, now = 0x1p-126f;
        if (id >= 0) {
          float* sc = (tid & 1 ? C.vscale : C.kscale) + (int64_t)id * C.H + h;
          if (pg == pf && old > 0) was = *sc;
          now = fmaxf(was, scale_for(__int_as_float(amax[tid])));
          if (now != was) *sc = now;
        }
        scales[pg][2 * (tid & 1)] = was;
        scales[pg][2 * (tid & 1) + 1] = now;
      }
      __syncthreads();
      // the page's earlier rows at raised scales (ratios are powers of two): all of
      // x, of v the groups that have no new ones
      if (old > 0 && ids[pf] >= 0) {
        const int64_t from = page_base(C, ids[pf], h);
        auto redo = [&](int8_t* at, int words, float f) {
          for (int i = tid; i < words; i += kThreads) {
            char4 q = *reinterpret_cast<char4*>(at + 4 * i);
            q.x = (signed char)rintf(q.x * f);
            q.y = (signed char)rintf(q.y * f);
            q.z = (signed char)rintf(q.z * f);
            q.w = (signed char)rintf(q.w * f);
            *reinterpret_cast<char4*>(at + 4 * i) = q;
          }
        };
        if (scales[pf][1] != scales[pf][0])
          redo(static_cast<int8_t*>(C.k) + from, old * D / 4, scales[pf][0] * recip2(scales[pf][1]));
        again = scales[pf][3] != scales[pf][2];
        if (again)
          redo(static_cast<int8_t*>(C.v) + from, old / kGroup * kGroup * D / 4,
               scales[pf][2] * recip2(scales[pf][3]));
      }
#pragma unroll
      for (int k = 0; k < kPass; ++k) {
        const int r = row0 + k * kStep, id = ids[r >> pshift];
        if (r < r0 || r >= r1 || id < 0) continue;
        const float rs = recip2(scales[r >> pshift][1]);
        float f[8];
        Vec16<bf16>::unpack(kept[k], f);
        const int64_t at = ((int64_t)id * C.H + h) * C.P + ((off0 + r) & pmask);
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(C.k) + at * D + dim0) =
            make_uint2(quant4(f[0], f[1], f[2], f[3], rs, odd), quant4(f[4], f[5], f[6], f[7], rs, odd));
      }
    }

    // v: warps take (group of 16 tokens, 16 dimensions) in turn
    constexpr int kSteps = D / 16;
    const int g0 = r0 / kGroup, g1 = (r1 - 1) / kGroup;
    for (int w = warp; w < (g1 - g0 + 1) * kSteps; w += kWarps) {
      const int rb = (g0 + w / kSteps) * kGroup, d0 = (w % kSteps) * 16;
      // tiles 0, 1: tokens {0,1,4,5,8,9,12,13} and {2,3,6,7,10,11,14,15} of
      // dimensions d0 ..; tiles 2, 3 the same of the next eight: lane (g, t) then
      // holds tokens 4t .. 4t + 3 of dimensions d0 + g and d0 + 8 + g
      const int i = lane & 7, tile = lane >> 3;
      const int trow = rb + (i >> 1) * 4 + (i & 1) + 2 * (tile & 1);
      uint32_t m[4];
      ldsm_x4_trans(m, vt + trow * kStride + d0 + 8 * (tile >> 1));
      const int id = ids[rb >> pshift];
      if (id < 0) continue;
      const int64_t at = (((int64_t)id * C.H + h) * C.P + ((off0 + rb) & pmask)) * D +
                         (d0 + (lane >> 2)) * kGroup + (lane & 3) * 4;
      const int tk = rb + (lane & 3) * 4;
      const bool all = tk >= r0 && tk + 4 <= r1;
      if constexpr (!I8) {
        bf16* dst = static_cast<bf16*>(C.v) + at;
#pragma unroll
        for (int k = 0; k < 2; ++k, dst += 8 * kGroup) {
          if (all) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(m[2 * k], m[2 * k + 1]);
          } else {
            uint16_t* e = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (tk + q >= r0 && tk + q < r1)
                e[q] = (uint16_t)(m[2 * k + (q >> 1)] >> (16 * (q & 1)));
          }
        }
      } else {
        int8_t* dst = static_cast<int8_t*>(C.v) + at;
        const float rs = recip2(scales[rb >> pshift][3]);
        const bool redo = again && tk < r0;
        const float vf = redo ? scales[rb >> pshift][2] * rs : 1.f;
        if (tk >= r1 || (tk + 4 <= r0 && !redo)) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k, dst += 8 * kGroup) {
          const uint32_t fresh = quant4(bf_lo(m[2 * k]), bf_hi(m[2 * k]), bf_lo(m[2 * k + 1]),
                                        bf_hi(m[2 * k + 1]), rs, odd);
          if (all) {
            *reinterpret_cast<uint32_t*>(dst) = fresh;
            continue;
          }
          char4 q = *reinterpret_cast<char4*>(dst);
          signed char* e = reinterpret_cast<signed char*>(&q);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (tk + j >= r0 && tk + j < r1) e[j] = (signed char)(fresh >> (8 * j));
            else if (tk + j < r0 && redo) e[j] = (signed char)rintf(e[j] * vf);
          }
          *reinterpret_cast<char4*>(dst) = q;
        }
      }
    }
    __syncthreads();  // the tile is free
    if (h + kBuf < h1) fetch(h + kBuf);
  }
}

struct GatherArgs {
  CacheView C;
  SeqTables S;
  bf16* x;
  bf16* v;
  int64_t xs[3], vs[3];
  int groups;  // groups of 16 positions that n rows can touch
};

// One warp: one group of 16 tokens of one head, back to rows. v is staged as
// bf16 in shared memory and read as transposed 8x8 tiles. Bound by DRAM: 68 us for
// 65536 int8 rows of 8 heads of 128 (0.91 of the copy rate; with each load used
// before the next is issued, and bytes widened by conversion instructions, 104).
// grid (groups / 8, heads, batch), block 256.
template <int D, bool I8>
__global__ void __launch_bounds__(256) k_cache_gather(GatherArgs A) {
  constexpr int kRow = kGroup + 8;  // padded shared row: 48 bytes
  __shared__ __align__(16) bf16 tile[8][D * kRow];
  const CacheView& C = A.C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  const int gi = blockIdx.x * 8 + warp;
  int len, nv;
  if (!seq_rows(A.S, C.P, b, &len, &nv) && blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    cache_error(C);
  if (gi >= A.groups) return;
  const int64_t at = (int64_t)(len / kGroup + gi) * kGroup;  // first position of the group
  const int i0 = (int)(at - len);                            // its row of the call
  bf16* xo = A.x + b * A.xs[0] + h * A.xs[1];
  bf16* vo = A.v + b * A.vs[0] + h * A.vs[1];
  int id = -1;
  if (max(i0, 0) < nv) {  // a sequence without rows has no group, wherever it starts
    id = page_of(C, A.S, b, (int)(at / C.P));
    if (id < 0 && lane == 0) cache_error(C);
  }
  if (id < 0) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int k = lane; k < kGroup * (D / 8); k += 32) {
      const int64_t i = i0 + k / (D / 8);
      if (i < 0 || i >= A.S.n) continue;
      *reinterpret_cast<uint4*>(xo + i * A.xs[2] + k % (D / 8) * 8) = z;
      *reinterpret_cast<uint4*>(vo + i * A.vs[2] + k % (D / 8) * 8) = z;
    }
    return;
  }
  const int64_t from = page_base(C, id, h) + (at & (C.P - 1)) * D;
  const int64_t hs = (int64_t)id * C.H + h;
  bf16* tl = tile[warp];
  // every load of the group before the first is used: 16 bytes of v, and of x
  // what makes 16 bytes of a row
  constexpr int kV = I8 ? D / 32 : D / 16, kK = D / 16;
  using Raw = std::conditional_t<I8, uint2, uint4>;
  uint4 vr[kV];
  Raw kr[kK];
  const unsigned char* vg = static_cast<const unsigned char*>(C.v) + from * (I8 ? 1 : 2);
  const unsigned char* kg = static_cast<const unsigned char*>(C.k) + from * (I8 ? 1 : 2);
#pragma unroll
  for (int k = 0; k < kV; ++k) vr[k] = *reinterpret_cast<const uint4*>(vg + (k * 32 + lane) * 16);
#pragma unroll
  for (int k = 0; k < kK; ++k) kr[k] = *reinterpret_cast<const Raw*>(kg + (k * 32 + lane) * sizeof(Raw));
  float ks = 1.f, vs = 1.f;
  if constexpr (I8) {
    ks = C.kscale[hs];
    vs = C.vscale[hs];
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    if constexpr (I8) {  // dimension 32 k + lane, 16 tokens
      const uint2 a = i8_values(vr[k].x, vs), b = i8_values(vr[k].y, vs);
      const uint2 c = i8_values(vr[k].z, vs), d = i8_values(vr[k].w, vs);
      *reinterpret_cast<uint4*>(tl + (k * 32 + lane) * kRow) = make_uint4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<uint4*>(tl + (k * 32 + lane) * kRow + 8) = make_uint4(c.x, c.y, d.x, d.y);
    } else {
      const int p = k * 32 + lane;
      *reinterpret_cast<uint4*>(tl + (p >> 1) * kRow + (p & 1) * 8) = vr[k];
    }
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int p = k * 32 + lane, r = p / (D / 8), piece = p % (D / 8);
    const int64_t i = i0 + r;
    if (i < 0 || i >= A.S.n) continue;
    uint4 u;
    if constexpr (I8) {
      const uint2 a = i8_values(kr[k].x, ks), b = i8_values(kr[k].y, ks);
      u = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      u = kr[k];
    }
    if (i >= nv) u = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(xo + i * A.xs[2] + piece * 8) = u;
  }
  __syncwarp();
  // tile j of a load: dimensions 8 t' + 2 j and + 1 (t' = 0..3) by eight tokens,
  // so that lane (g, t) gathers dimensions 8 t .. 8 t + 7 of token g
#pragma unroll
  for (int st = 0; st < D / 32 * 2; ++st) {
    const int dim0 = (st >> 1) * 32, tok0 = (st & 1) * 8;
    const int i = lane & 7, j = lane >> 3;
    uint32_t m[4];
    ldsm_x4_trans(m, tl + (dim0 + 8 * (i >> 1) + 2 * j + (i & 1)) * kRow + tok0);
    const int64_t row = i0 + tok0 + (lane >> 2);
    if (row < 0 || row >= A.S.n) continue;
    *reinterpret_cast<uint4*>(vo + row * A.vs[2] + dim0 + (lane & 3) * 8) =
        row < nv ? make_uint4(m[0], m[1], m[2], m[3]) : make_uint4(0, 0, 0, 0);
  }
}

}  // namespace lsh
