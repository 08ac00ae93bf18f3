// Shared-QK attention of a sequence's newest tokens over the paged cache.
//
// Row t at position p = len + t sees the cached tokens j <= p:
//   l_j = x_t . k_j / (||x_j|| sqrt(d)),  l_p = -1e5,
//   out = sum_j softmax(l)_j v_j,  lse = ln sum_j exp l_j.
// With one row, or a handful, for every sequence and head, each cached byte is
// used once: the kernel is a stream through the cache and is bound by DRAM.
//
// Work. A unit is a tile of 128 tokens for one (sequence, head, eight rows).
// Units are numbered through sequences, heads, row groups and tiles, and the
// blocks (one or two an SM, persistent) take equal runs of them, so that the
// card is evenly loaded whatever the lengths are: they are read on the device.
// A (sequence, head) that several blocks share leaves partial sums in the
// workspace, which k_cache_combine joins in a fixed order.
//
// Block. One warp walks the units, looks pages up a batch of four tiles ahead
// and issues bulk copies into a ring of shared-memory stages; eight warps
// compute, each on 16 tokens of every tile, without a barrier among them until
// a (sequence, head) ends. S = Q K^T and O += P V are warp products
// (m16n8k16): eight rows do not fill a tcgen05 tile, and the tensor work is a
// tenth of what the warp instructions can do at DRAM speed. The contraction
// index may be permuted at will as long as both operands agree, so each lane
// takes the dimensions (of K) and the tokens (of V, whose groups lie dimension
// by dimension in the cache) that are consecutive in memory, and feeds them to
// the product as they are: no transposes, no shuffles. The 16 rows of a product
// hold the eight rows twice: weights as high and low parts (bf16: 2^-17, f16:
// 2^-22 together), so that P V loses nothing against fp32 weights. int8 keys and
// values are exact in f16; rows of x in f16, scaled by a power of two, also as
// high and low part.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "cache.cuh"

namespace lsh {

constexpr int kTileTok = 128;   // tokens of a unit
constexpr int kAttWarps = 8;    // computing warps, 16 tokens of a unit each
constexpr int kAttThreads = 32 * (kAttWarps + 1);
constexpr int kAttRows = 8;     // rows of a unit
constexpr float kLog2e = 1.4426950408889634f;

struct AttendArgs {
  CacheView C;
  SeqTables S;
  const bf16* x;
  bf16* out;
  float* lse;
  int64_t xs[3], os[3];
  float* part;     // [grid][2][8][D] unnormalised sums of split units
  float* part_ml;  // [grid][2][8][2] their maxima (log2) and weights' sums
  int* rec;        // [grid][8]: the split (sequence, head) that starts in a block
};

// A ring stage's header, written by the copying warp.
struct TileMeta {
  int b, h, q0, rows;   // first row of the group and how many
  int len, vis, t0;     // tokens before the rows; tokens they see; first of the tile
  int flags, slot;      // kFirst | kLast | kWhole | kEnd; partial slot
  uint32_t ok;          // bit s: tokens 16 s .. of the tile are there
  float ks[8], vs[8];   // scales of these (int8)
};
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8;

template <int D, bool I8>
struct AttCfg {
  static constexpr int E = I8 ? 1 : 2;
  static constexpr int kK = kTileTok * D * E;
  static constexpr int kNorm = kTileTok * 4;
  static constexpr int kQ = kAttRows * D * 2;
  static constexpr int kMeta = 256;
  static constexpr int kStage = 2 * kK + kNorm + kQ + kMeta;
  // as many stages as two blocks an SM (D 64) or one (D 128) have room for
  static constexpr int kBlocks = D == 64 ? 2 : 1;
  static constexpr int kMerge = 4 * kAttRows * D * 4;  // four warps' sums
  static constexpr int kFixed = kMerge + 1024;
  static constexpr int kRoom = (kBlocks == 2 ? 113 * 1024 : 226 * 1024) - kFixed;
  static constexpr int kStages = kRoom / kStage < 6 ? kRoom / kStage : 6;
  static constexpr int kSmem = kFixed + kStages * kStage;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, bf16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four int8 to two pairs of f16: 1024 + (q + 128) is written into the mantissa
// and 1152 taken off, both exact.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t* b0, uint32_t* b1) {
  w ^= 0x80808080u;
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
  __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), off);
  __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
  *b0 = *reinterpret_cast<uint32_t*>(&a);
  *b1 = *reinterpret_cast<uint32_t*>(&b);
}

// (x, y) as a pair of T and what the pair leaves over, as another.
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo, bf16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const __nv_bfloat162 l =
      __floats2bfloat162_rn(x - __bfloat162float(h.x), y - __bfloat162float(h.y));
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo, __half) {
  const __half2 h = __floats2half2_rn(x, y);
  const __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Units of sequence b: heads x row groups x tiles.
__device__ __forceinline__ int64_t att_units(int H, int len, int nv) {
  const int groups = (nv + kAttRows - 1) / kAttRows;
  const int tiles = (int)(((int64_t)len + nv + kTileTok - 1) / kTileTok);
  return (int64_t)H * groups * tiles;
}

// ------------------------------------------------------------- the copying warp
// Where the walk over the units stands.
struct UnitCursor {
  int b, h, grp, tile;       // the next unit
  int groups, tiles, len, nv;  // of its sequence
};

template <int D, bool I8>
__device__ void att_copy_warp(const AttendArgs& A, unsigned char* stages, uint64_t* full,
                              uint64_t* empty) {
  using Cfg = AttCfg<D, I8>;
  const CacheView& C = A.C;
  const SeqTables& S = A.S;
  const int lane = threadIdx.x & 31;
  const unsigned kAll = 0xffffffffu;

  // all units, then this block's run of them
  int64_t N = 0;
  for (int base = 0; base < S.B; base += 32) {
    int len = 0, nv = 0;
    if (base + lane < S.B) seq_rows(S, C.P, base + lane, &len, &nv);
    N += att_units(C.H, len, nv);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) N += __shfl_xor_sync(kAll, N, o);
  const int64_t G = min((int64_t)gridDim.x, N);
  int64_t u = 0, u1 = 0;
  if ((int64_t)blockIdx.x < G) {
    u = N * blockIdx.x / G;
    u1 = N * (blockIdx.x + 1) / G;
  }
  const int64_t u0 = u;

  // the sequence that holds unit u; lens of 32 sequences are kept in the lanes
  int wbase = 0, wlen = 0, wnv = 0;
  UnitCursor c{};
  if (u < u1) {
    int64_t before = 0;
    for (;; wbase += 32) {
      wlen = wnv = 0;
      if (wbase + lane < S.B) seq_rows(S, C.P, wbase + lane, &wlen, &wnv);
      const int64_t mine = att_units(C.H, wlen, wnv);
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned past = __ballot_sync(kAll, before + incl > u);
      if (past) {
        const int l = __ffs(past) - 1;
        const int64_t at = u - (before + __shfl_sync(kAll, incl - mine, l));
        c.b = wbase + l;
        c.len = __shfl_sync(kAll, wlen, l);
        c.nv = __shfl_sync(kAll, wnv, l);
        c.groups = (c.nv + kAttRows - 1) / kAttRows;
        c.tiles = (int)(((int64_t)c.len + c.nv + kTileTok - 1) / kTileTok);
        c.tile = (int)(at % c.tiles);
        const int64_t hg = at / c.tiles;
        c.grp = (int)(hg % c.groups);
        c.h = (int)(hg / c.groups);
        break;
      }
      before += __shfl_sync(kAll, incl, 31);
    }
  }
  int seg_from_zero = c.tile == 0;  // this block has the segment's first tile
  int rec_valid = 0, rec_count = 0;

  // lanes 8 i .. 8 i + 7 hold tile i of a batch: lane 8 i + s its tokens 16 s ..
  struct Batch {
    int n;  // tiles (the same in all lanes)
    int b, h, q0, rows, len, vis, t0, flags, slot;
    int id;
    float ks, vs;
  };
  const int grp_of = lane >> 3, sl = lane & 7;
  int last_b = 0, last_h = 0, last_q0 = 0, last_rows = 0;

  auto next_batch = [&](Batch& m) {
    m.n = 0;
    m.id = -1;
    m.vis = m.t0 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (u >= u1) break;
      const int q0 = c.grp * kAttRows, rows = min(kAttRows, c.nv - q0);
      const bool first = u == u0 || c.tile == 0;
      if (first) seg_from_zero = c.tile == 0;
      const bool ends = c.tile == c.tiles - 1;
      const bool last = ends || u == u1 - 1;
      if (grp_of == i) {
        m.b = c.b;
        m.h = c.h;
        m.q0 = q0;
        m.rows = rows;
        m.len = c.len;
        m.vis = c.len + q0 + rows;
        m.t0 = c.tile * kTileTok;
        m.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (ends && seg_from_zero ? kWhole : 0);
        m.slot = seg_from_zero;
      }
      if (u == u1 - 1 && seg_from_zero && !ends) {
        // the segment goes on in the blocks behind: how many
        const int64_t end = u + (c.tiles - 1 - c.tile);
        rec_valid = 1;
        rec_count = (int)(((end + 1) * G - 1) / N) - (int)blockIdx.x + 1;
        last_b = c.b;
        last_h = c.h;
        last_q0 = q0;
        last_rows = rows;
      }
      ++m.n;
      ++u;
      if (++c.tile == c.tiles) {
        c.tile = 0;
        if (++c.grp == c.groups) {
          c.grp = 0;
          if (++c.h == C.H && u < u1) {
            c.h = 0;
            do {  // the next sequence with rows
              ++c.b;
              if (c.b == wbase + 32) {
                wbase += 32;
                wlen = wnv = 0;
                if (wbase + lane < S.B) seq_rows(S, C.P, wbase + lane, &wlen, &wnv);
              }
              c.nv = __shfl_sync(kAll, wnv, c.b - wbase);
            } while (c.nv == 0);
            c.len = __shfl_sync(kAll, wlen, c.b - wbase);
            c.groups = (c.nv + kAttRows - 1) / kAttRows;
            c.tiles = (int)(((int64_t)c.len + c.nv + kTileTok - 1) / kTileTok);
          }
        }
      }
    }
    const int pos = m.t0 + 16 * sl;
    if (grp_of < m.n && pos < m.vis) {
      m.id = page_of(C, S, m.b, pos / C.P);
      if (m.id < 0) cache_error(C);
    }
  };
  auto scales = [&](Batch& m) {
    m.ks = m.vs = 0.f;
    if constexpr (I8)
      if (m.id >= 0) {
        const int64_t hs = (int64_t)m.id * C.H + m.h;
        m.ks = C.kscale[hs];
        m.vs = C.vscale[hs];
      }
  };

  int st = 0;
  uint32_t ph = 0;
  bool good = true;
  const int chunk = min(C.P / 16, 8);  // 16-token pieces that one copy takes
  auto issue = [&](const Batch& m, int i) {
    if (!good) return;
    good = sm100::mbar_wait(&empty[st], ph ^ 1);
    if (!good) return;
    unsigned char* sp = stages + (size_t)st * Cfg::kStage;
    TileMeta* mt = reinterpret_cast<TileMeta*>(sp + 2 * Cfg::kK + Cfg::kNorm + Cfg::kQ);
    const bool mine = grp_of == i;
    const unsigned ok = __ballot_sync(kAll, mine && m.id >= 0);
    if (mine) {
      if constexpr (I8) {
        mt->ks[sl] = m.ks;
        mt->vs[sl] = m.vs;
      }
      if (sl == 0) {
        mt->b = m.b;
        mt->h = m.h;
        mt->q0 = m.q0;
        mt->rows = m.rows;
        mt->len = m.len;
        mt->vis = m.vis;
        mt->t0 = m.t0;
        mt->flags = m.flags;
        mt->slot = m.slot;
        mt->ok = ok >> (8 * i);
      }
    }
    __syncwarp();
    if (mine && sl == 0)
      sm100::mbar_expect_tx(&full[st], __popc(ok) * (32 * D * Cfg::E + 64) +
                                           (m.flags & kFirst ? m.rows * D * 2 : 0));
    __syncwarp();
    if (mine) {
      if (sl % chunk == 0 && m.id >= 0) {
        const int pos = m.t0 + 16 * sl;
        const int n = min(chunk, (m.vis - pos + 15) / 16);
        const int64_t from = (page_base(C, m.id, m.h) + (int64_t)(pos % C.P) * D) * Cfg::E;
        const uint32_t bytes = n * 16 * D * Cfg::E;
        sm100::bulk_copy_g2s(sp + sl * 16 * D * Cfg::E, static_cast<char*>(C.k) + from, bytes,
                             &full[st]);
        sm100::bulk_copy_g2s(sp + Cfg::kK + sl * 16 * D * Cfg::E, static_cast<char*>(C.v) + from,
                             bytes, &full[st]);
        sm100::bulk_copy_g2s(sp + 2 * Cfg::kK + sl * 64,
                             C.kinv + ((int64_t)m.id * C.H + m.h) * C.P + pos % C.P, n * 64,
                             &full[st]);
      }
      if ((m.flags & kFirst) && sl < m.rows)
        sm100::bulk_copy_g2s(sp + 2 * Cfg::kK + Cfg::kNorm + sl * D * 2,
                             A.x + m.b * A.xs[0] + m.h * A.xs[1] + (int64_t)(m.q0 + sl) * A.xs[2],
                             D * 2, &full[st]);
    }
    __syncwarp();
    if (++st == Cfg::kStages) {
      st = 0;
      ph ^= 1;
    }
  };

  Batch cur, nxt;
  next_batch(cur);
  scales(cur);
  while (cur.n > 0) {
    // the next batch's page numbers travel while this batch's copies are
    // issued, its scales behind the second half of them
    next_batch(nxt);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < cur.n) issue(cur, i);
    scales(nxt);
#pragma unroll
    for (int i = 2; i < 4; ++i)
      if (i < cur.n) issue(cur, i);
    cur = nxt;
  }
  if (good) good = sm100::mbar_wait(&empty[st], ph ^ 1);
  if (good) {
    if (lane == 0) {
      reinterpret_cast<TileMeta*>(stages + (size_t)st * Cfg::kStage + 2 * Cfg::kK + Cfg::kNorm +
                                  Cfg::kQ)->flags = kEnd;
      sm100::mbar_arrive(&full[st]);
    }
  } else {
    if (lane == 0 && C.status) record_status(C.status, 5u /* LSH_ERR_TIMEOUT */);
    // let every copy land before the block's memory goes away
    for (int i = 0; i < Cfg::kStages; ++i) {
      if (++st == Cfg::kStages) st = 0;
      sm100::mbar_wait(&full[st], 0, 100000000ull);
      sm100::mbar_wait(&full[st], 1, 100000000ull);
    }
  }
  if (lane == 0) {
    int* r = A.rec + blockIdx.x * 8;
    r[0] = rec_valid;
    r[1] = rec_count;
    r[2] = last_b;
    r[3] = last_h;
    r[4] = last_q0;
    r[5] = last_rows;
  }
}

// ------------------------------------------------------------- the computing warps
// Rows past a sequence's own are zeros, their lse -inf; sequences are shared
// out over the blocks.
template <int D>
__device__ void att_pad_rows(const AttendArgs& A) {
  for (int b = blockIdx.x; b < A.S.B; b += gridDim.x) {
    int len, nv;
    if (!seq_rows(A.S, A.C.P, b, &len, &nv) && threadIdx.x == 0) cache_error(A.C);
    const int64_t pad = (int64_t)(A.S.n - nv) * A.C.H;
    for (int64_t i = threadIdx.x; i < pad * (D / 8); i += kAttWarps * 32) {
      const int64_t r = i / (D / 8);
      const int h = (int)(r % A.C.H), t = nv + (int)(r / A.C.H);
      *reinterpret_cast<uint4*>(A.out + b * A.os[0] + h * A.os[1] + t * A.os[2] +
                                i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
      if (i % (D / 8) == 0) A.lse[((int64_t)b * A.C.H + h) * A.S.n + t] = -INFINITY;
    }
  }
}

template <int D, bool I8>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D, I8>::kBlocks) k_cache_attend(AttendArgs A) {
  using Cfg = AttCfg<D, I8>;
  using T = std::conditional_t<I8, __half, bf16>;
  constexpr int kSteps = D / 16;  // 16-wide steps of Q K^T
  constexpr int kN = D / 8;       // 8-wide column tiles of P V
  extern __shared__ __align__(16) unsigned char smem[];
  float* merge = reinterpret_cast<float*>(smem);  // [4][8][D]
  float* wm = reinterpret_cast<float*>(smem + Cfg::kMerge);  // [8 warps][8 rows]
  float* wl = wm + 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(wl + 64);
  uint64_t* empty = full + 8;
  unsigned char* stages = smem + Cfg::kFixed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], kAttWarps);
    }
    sm100::fence_mbar_init();
  }
  __syncthreads();
  if (warp == kAttWarps) {
    att_copy_warp<D, I8>(A, stages, full, empty);
    return;
  }
  att_pad_rows<D>(A);

  const float cs = kLog2e / sqrtf((float)D);
  // Q as A operand: step s, a0 and a2 (row g); int8: a1 and a3 their low parts
  uint32_t qh[2 * kSteps], ql[I8 ? 2 * kSteps : 1];
  float o[kN][4];
  float m = -INFINITY, l = 0.f, qscale = 1.f;
  float vref = 0.f, vinv = 0.f;  // int8: o counts in units of the scale vref
  int st = 0;
  uint32_t ph = 0;
  bool good = true;

  for (;;) {
    good = sm100::mbar_wait(&full[st], ph);
    if (!good) {
      if (lane == 0 && A.C.status) record_status(A.C.status, 5u /* LSH_ERR_TIMEOUT */);
      sm100::bar_sync_any(1, kAttWarps * 32, true);
      return;
    }
    const unsigned char* sp = stages + (size_t)st * Cfg::kStage;
    const TileMeta* mt = reinterpret_cast<const TileMeta*>(sp + 2 * Cfg::kK + Cfg::kNorm + Cfg::kQ);
    const int flags = mt->flags;
    if (flags & kEnd) {
      sm100::bar_sync_any(1, kAttWarps * 32, false);
      break;  // k_cache_combine may be brought in
    }
    if (flags & kFirst) {
      const unsigned char* qp = sp + 2 * Cfg::kK + Cfg::kNorm + g * D * 2;
      if constexpr (I8) {
        // dimensions 64 j + 16 t .. + 15 of row g: steps 4 j .. 4 j + 3
        float f[D / 4];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          Vec16<bf16>::unpack(*reinterpret_cast<const uint4*>(qp + (64 * j + 16 * t) * 2), f + 16 * j);
          Vec16<bf16>::unpack(*reinterpret_cast<const uint4*>(qp + (64 * j + 16 * t + 8) * 2), f + 16 * j + 8);
        }
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(f[i]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // a power of two that brings the row's largest value to [1, 2)
        int e = (int)((__float_as_uint(top) >> 23) & 255) - 127;
        e = max(-126, min(126, e));
        qscale = __uint_as_float((uint32_t)(e + 127) << 23);
        const float up = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) split2(f[2 * i] * up, f[2 * i + 1] * up, &qh[i], &ql[i], T());
      } else {
        // dimensions 32 j + 8 t .. + 7: steps 2 j and 2 j + 1
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(qp + (32 * j + 8 * t) * 2);
          qh[4 * j] = u.x;
          qh[4 * j + 1] = u.y;
          qh[4 * j + 2] = u.z;
          qh[4 * j + 3] = u.w;
        }
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
      m = -INFINITY;
      l = 0.f;
      vref = 0.f;
    }

    const int pos0 = mt->t0 + 16 * warp;  // this warp's 16 tokens
    if (mt->ok >> warp & 1) {
      // S: column c of half j is token 4 (c / 2) + 2 j + c % 2, so that this lane
      // holds tokens 4 t .. 4 t + 3 of row g
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
        const unsigned char* kp =
            sp + (16 * warp + 4 * (g >> 1) + 2 * j + (g & 1)) * D * Cfg::E + 16 * t;
#pragma unroll
        for (int i = 0; i < D * Cfg::E / 64; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(kp + 64 * i);
          if constexpr (I8) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t b0, b1;
              i8_to_f16(w[k], &b0, &b1);
              const int a = 2 * (4 * i + k);
              mma_16816(s[j], qh[a], ql[a], qh[a + 1], ql[a + 1], b0, b1, T());
            }
          } else {
            mma_16816(s[j], qh[4 * i], 0u, qh[4 * i + 1], 0u, u.x, u.y, T());
            mma_16816(s[j], qh[4 * i + 2], 0u, qh[4 * i + 3], 0u, u.z, u.w, T());
          }
        }
      }
      const float4 kn = *reinterpret_cast<const float4*>(sp + 2 * Cfg::kK + (16 * warp + 4 * t) * 4);
      float f = cs;
      if constexpr (I8) f *= mt->ks[warp] * qscale;
      float p[4];
      p[0] = (s[0][0] + s[0][2]) * (kn.x * f);
      p[1] = (s[0][1] + s[0][3]) * (kn.y * f);
      p[2] = (s[1][0] + s[1][2]) * (kn.z * f);
      p[3] = (s[1][1] + s[1][3]) * (kn.w * f);
      const int self = mt->len + mt->q0 + g - (pos0 + 4 * t);  // row g's own token
      const bool tail = pos0 + 16 > mt->len + mt->q0;
      if (tail) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          p[k] = k > self ? -INFINITY : k == self ? kSelfLogit * kLog2e : p[k];
      }
      float top = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const float mn = fmaxf(m, top);
      float corr = 1.f;
      if (mn > m) corr = ex2(m - mn);
      float ratio = 1.f;
      bool again = mn > m;
      if constexpr (I8) {
        const float vs = mt->vs[warp];
        if (vs > vref) {
          corr *= vref * (1.f / vs);
          vref = vs;
          vinv = 1.f / vs;
          again = true;
        }
        ratio = vs * vinv;
      }
      if (__any_sync(~0u, again)) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] *= corr;
      }
      if (mn > m) l *= ex2(m - mn);
      m = mn;
      const float ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = ex2(p[k] - ref);
        l += p[k];
        if constexpr (I8) p[k] *= ratio;
      }
      uint32_t a[4];
      split2(p[0], p[1], &a[0], &a[1], T());
      split2(p[2], p[3], &a[2], &a[3], T());
      const unsigned char* vp = sp + Cfg::kK + 16 * warp * D * Cfg::E + (g * 16 + 4 * t) * Cfg::E;
      if (I8 || !tail) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          uint32_t b0, b1;
          if constexpr (I8) {
            i8_to_f16(*reinterpret_cast<const uint32_t*>(vp + i * 128), &b0, &b1);
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vp + i * 256);
            b0 = u.x;
            b1 = u.y;
          }
          mma_16816(o[i], a[0], a[1], a[2], a[3], b0, b1, T());
        }
      } else {
        // values that some row of the group must not see: slots behind the last
        // row hold anything, a later row's value may be infinite, and 0 times it
        // is NaN. Those behind are cleared; where one in between is not finite,
        // the tokens go one by one and each row takes its own only.
        const int behind = mt->vis - (pos0 + 4 * t);  // tokens of this lane that count
        const uint32_t k0 = behind >= 2 ? ~0u : behind == 1 ? 0xffffu : 0u;
        const uint32_t k1 = behind >= 4 ? ~0u : behind == 3 ? 0xffffu : 0u;
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint2 u = *reinterpret_cast<const uint2*>(vp + i * 256);
          const uint32_t w[2] = {u.x & k0, u.y & k1};
#pragma unroll
          for (int k = 0; k < 2; ++k)
            odd |= (uint32_t)((w[k] & 0x7f80u) == 0x7f80u) | (uint32_t)((w[k] & 0x7f800000u) == 0x7f800000u);
        }
        if (!__any_sync(~0u, odd)) {
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const uint2 u = *reinterpret_cast<const uint2*>(vp + i * 256);
            mma_16816(o[i], a[0], a[1], a[2], a[3], u.x & k0, u.y & k1, T());
          }
        } else {
          for (int j = 0; j < 16; ++j) {
            const bool mine = j >> 2 == t;
            const uint32_t half = j & 1 ? 0xffff0000u : 0xffffu;
            const uint32_t e0 = mine && !(j & 2) ? half & k0 : 0u, e1 = mine && j & 2 ? half & k1 : 0u;
            const bool sees = pos0 + j <= mt->len + mt->q0 + g;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const uint2 u = *reinterpret_cast<const uint2*>(vp + i * 256);
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816(d, a[0], a[1], a[2], a[3], u.x & e0, u.y & e1, T());
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (sees) o[i][k] += d[k];
            }
          }
        }
      }
    }

    if (flags & kLast) {
      // join the eight warps: maxima, then sums scaled to the common one
      l += __shfl_xor_sync(~0u, l, 1);
      l += __shfl_xor_sync(~0u, l, 2);
      if (t == 0) wm[warp * 8 + g] = m;
      if (sm100::bar_sync_any(1, kAttWarps * 32, false)) return;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, wm[w * 8 + g]);
      const float f = m == -INFINITY && !(l != l) ? 0.f : ex2(m - (M == -INFINITY ? 0.f : M));
      if (t == 0) wl[warp * 8 + g] = m == -INFINITY && l == 0.f ? 0.f : l * f;
      const float fo = I8 ? f * vref : f;
      float* mine = merge + ((warp & 3) * 8 + g) * D + 2 * t;
      if (warp >= 4) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          *reinterpret_cast<float2*>(mine + 8 * i) =
              make_float2((o[i][0] + o[i][2]) * fo, (o[i][1] + o[i][3]) * fo);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (warp < 4) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float2 e = *reinterpret_cast<float2*>(mine + 8 * i);
          *reinterpret_cast<float2*>(mine + 8 * i) = make_float2(
              (o[i][0] + o[i][2]) * fo + e.x, (o[i][1] + o[i][3]) * fo + e.y);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      // a warp takes a row: lane's D / 32 dimensions
      const int rows = mt->rows;
      if (warp < rows) {
        constexpr int DL = D / 32;
        float sum[DL], L = 0.f, Mr = -INFINITY;
#pragma unroll
        for (int k = 0; k < DL; ++k) sum[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
          L += wl[w * 8 + warp];
          Mr = fmaxf(Mr, wm[w * 8 + warp]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int k = 0; k < DL; ++k) sum[k] += merge[(w * 8 + warp) * D + lane * DL + k];
        if (flags & kWhole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          alignas(8) bf16 e[DL];
#pragma unroll
          for (int k = 0; k < DL; ++k) e[k] = __float2bfloat16_rn(sum[k] * inv);
          bf16* op = A.out + mt->b * A.os[0] + mt->h * A.os[1] + (int64_t)(mt->q0 + warp) * A.os[2] + lane * DL;
          if constexpr (DL == 4) *reinterpret_cast<uint2*>(op) = *reinterpret_cast<uint2*>(e);
          else *reinterpret_cast<uint32_t*>(op) = *reinterpret_cast<uint32_t*>(e);
          if (lane == 0)
            A.lse[((int64_t)mt->b * A.C.H + mt->h) * A.S.n + mt->q0 + warp] =
                L == 0.f ? -INFINITY : (Mr + log2f(L)) * 0.6931471805599453f;
        } else {
          const int64_t row = ((int64_t)blockIdx.x * 2 + mt->slot) * 8 + warp;
#pragma unroll
          for (int k = 0; k < DL; ++k) A.part[row * D + lane * DL + k] = sum[k];
          if (lane == 0) {
            A.part_ml[row * 2] = Mr;
            A.part_ml[row * 2 + 1] = L;
          }
        }
      }
      // the buffers are written again only behind the next segment's first barrier,
      // but wm before it
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&empty[st]);
    if (++st == Cfg::kStages) {
      st = 0;
      ph ^= 1;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the parts of a (sequence, head, row) that several blocks of
// k_cache_attend have left: block i's last one, then the first of each block
// behind it, in this order whatever runs when.
// grid (blocks of k_cache_attend, 8 rows), block 128.
template <int D>
__global__ void __launch_bounds__(128) k_cache_combine(AttendArgs A) {
  constexpr int DL = D / 32;
  // launched while k_cache_attend still runs: wait for its end, and its writes
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* r = A.rec + blockIdx.x * 8;
  const int row = blockIdx.y;
  if (!r[0] || row >= r[5]) return;
  const int count = r[1], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float sm[4], sl[4], so[4][D];
  // parts of this warp: running maximum, then a second pass
  float M = -INFINITY;
  for (int j = threadIdx.x; j < count; j += 128) {
    const int64_t p = ((int64_t)(blockIdx.x + j) * 2 + (j == 0)) * 8 + row;
    M = fmaxf(M, A.part_ml[p * 2]);
  }
  M = warp_max(M);
  if (lane == 0) sm[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) o[k] = 0.f;
#pragma unroll 4
  for (int j = warp; j < count; j += 4) {
    const int64_t p = ((int64_t)(blockIdx.x + j) * 2 + (j == 0)) * 8 + row;
    const float f = ex2(A.part_ml[p * 2] - ref);
    L += A.part_ml[p * 2 + 1] * f;
#pragma unroll
    for (int k = 0; k < DL; ++k) o[k] += A.part[p * D + lane * DL + k] * f;
  }
  if (lane == 0) sl[warp] = L;
#pragma unroll
  for (int k = 0; k < DL; ++k) so[warp][lane * DL + k] = o[k];
  __syncthreads();
  L = sl[0] + sl[1] + sl[2] + sl[3];
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int b = r[2], h = r[3], t = r[4] + row;
  for (int dim = threadIdx.x; dim < D; dim += 128)
    A.out[b * A.os[0] + h * A.os[1] + t * A.os[2] + dim] =
        __float2bfloat16_rn((so[0][dim] + so[1][dim] + so[2][dim] + so[3][dim]) * inv);
  if (threadIdx.x == 0)
    A.lse[((int64_t)b * A.C.H + h) * A.S.n + t] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace lsh
