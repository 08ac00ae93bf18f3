// Shared-QK attention of a sequence's newest tokens over the paged cache.
//
// Row t at position p = len + t sees the cached tokens j <= p:
//   l_j = x_t . k_j / (||x_j|| sqrt(d)),  l_p = -1e5,
//   out = sum_j softmax(l)_j v_j,  lse = ln sum_j exp l_j.
// With one row, or a handful, for every sequence and head, each cached byte is
// used once: the kernel is a stream through the cache and is bound by DRAM.
//
// Work. A unit is 64 tokens (int8) or 32 (bf16) for one (sequence, head, eight
// rows): a segment. Units are numbered through sequences, heads, row groups and
// tokens, and the blocks (persistent, one or two an SM) take equal runs of them,
// so that the card is evenly loaded whatever the lengths are: they are read on
// the device. A segment that several blocks share leaves partial sums in the
// workspace, which k_cache_combine joins in a fixed order.
//
// Block. Two warps walk the units, look the pages of the next ones up while they
// issue the copies of these, and fill a ring of shared-memory stages, one unit
// each, by bulk copies; eight warps compute, unit n by warp n % 8. They meet only
// where a segment ends of which the block had more than one unit.
//
// S = Q K^T and O += P V are warp products (m16n8k16): eight rows do not fill a
// tcgen05 tile, and DRAM allows ten times the tensor work. A contraction's index
// may be permuted at will as long as both operands agree, so a lane takes the
// dimensions of K (and the tokens of V, whose groups lie dimension by dimension
// in the cache) that are consecutive in memory, by 16 bytes, and feeds them to
// the products as they are: no transposes, no shuffles. The 16 rows of P hold the
// weights of eight as high and low parts (2^-17 together in bf16, 2^-22 in f16),
// so that P V loses nothing against fp32 weights (int8: those below 2^-39 of a
// row's largest are dropped). int8 keys and values are exact
// in f16. There the rows of x are f16 too, scaled by a power of two to a largest
// value in [1, 2): exact but for values below 2^-17 of it, which are off by 2^-25.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "cache.cuh"

namespace lsh {

constexpr int kAttWarps = 8;    // computing warps
constexpr int kAttThreads = 32 * (kAttWarps + 2);
constexpr int kAttRows = 8;     // rows of a segment
constexpr int kSegRing = 32;    // more than the segments that stages can hold
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
struct UnitMeta {
  int b, h, q0, rows;   // the segment's first row and how many
  int len, t0;          // tokens before the sequence's rows; the unit's first
  int vis;              // tokens that the segment's last row sees
  int flags, slot;      // kRows ...; slot of a partial result
  int joins;            // segments that have to be joined before this unit
  int n;                // the unit's number in the block
  uint32_t ok;          // bit s: tokens 16 s .. of the unit are there
  float ks[4], vs[4];   // their scales (int8)
};
// brings the segment's rows (the first eight units: a warp's first); the block's
// only unit of it; all of the segment is the block's; nothing follows
constexpr int kRows = 1, kSolo = 2, kWhole = 4, kEnd = 8;

struct SegInfo {  // of a segment that warps join
  int b, h, q0, rows, whole, slot;
};

template <int D, bool I8>
struct AttCfg {
  static constexpr int E = I8 ? 1 : 2;
  static constexpr int kGroups = I8 ? 4 : 2;        // 16-token groups of a unit
  static constexpr int kTok = 16 * kGroups;
  static constexpr int kK = kTok * D * E;
  // groups of v are set apart by 32 (64) bytes: the 16-byte pieces that eight
  // lanes read together then lie in different banks
  static constexpr int kVGroup = 16 * D * E + (I8 ? 32 : 64);
  static constexpr int kNorm = kK + kGroups * kVGroup;  // offsets in a stage
  static constexpr int kX = kNorm + kTok * 4;
  static constexpr int kMeta = kX + kAttRows * D * 2;
  static constexpr int kStage = kMeta + 128;
  // two blocks an SM where their registers allow it
  static constexpr int kBlocks = D == 64 ? 2 : 1;
  static constexpr int kMerge = 4 * kAttRows * D * 4;  // four warps' sums
  static constexpr int kFixed = kMerge + 2048;
  static constexpr int kRoom = (kBlocks == 2 ? 113 * 1024 : 226 * 1024) - kFixed;
  // even: a stage's units then have one parity, and come from one copying warp,
  // which has seen the stage freed every time
  static constexpr int kStages = (kRoom / kStage < 16 ? kRoom / kStage : 16) & ~1;
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

// ------------------------------------------------------------- the copying warp
// A sequence's row groups and units of a segment of it.
template <int kTok>
__device__ __forceinline__ int64_t att_units(int H, int len, int nv, int* groups, int* units) {
  *groups = (nv + kAttRows - 1) / kAttRows;
  *units = (int)(((int64_t)len + nv + kTok - 1) / kTok);
  return (int64_t)H * *groups * *units;
}

// Wait until unit n is in its stage. The stage's units belong to different warps,
// so the phase alone does not tell: a warp that comes early would take the unit
// before the last one's for its own. The number in the header is written after
// the stage has been freed, and the phase is the right one from then on.
__device__ __forceinline__ bool att_wait_unit(const UnitMeta* mt, uint64_t* full, uint32_t ph, int n) {
  const volatile int* at = &mt->n;
  if (*at != n) {
    const uint64_t t0 = sm100::global_ns();
    while (*at != n) {
      __nanosleep(40);
      if (sm100::global_ns() - t0 > sm100::kWaitLimitNs) return false;
    }
  }
  return sm100::mbar_wait(full, ph);
}

// Two warps copy: warp `par` the units n of its parity (one cannot issue a unit
// every 370 ns, which is what DRAM allows). Both walk all of them.
template <int D, bool I8>
__device__ void att_copy_warp(const AttendArgs& A, unsigned char* stages, uint64_t* full,
                              uint64_t* empty, SegInfo* segs, int par) {
  using Cfg = AttCfg<D, I8>;
  constexpr int NG = Cfg::kGroups, kBatch = 32 / NG;
  const CacheView& C = A.C;
  const SeqTables& S = A.S;
  const int lane = threadIdx.x & 31;
  const unsigned kAll = 0xffffffffu;
  const int pshift = __ffs(C.P) - 1;

  // the tokens of 32 sequences are kept in the lanes; all units, and this
  // block's run of them
  int wbase = 0, wlen = 0, wnv = 0;
  auto window = [&](int base) {
    wbase = base;
    wlen = wnv = 0;
    if (base + lane < S.B) seq_rows(S, C.P, base + lane, &wlen, &wnv);
  };
  int groups, units;
  int64_t N = 0;
  for (int base = 0; base < S.B; base += 32) {
    window(base);
    N += att_units<Cfg::kTok>(C.H, wlen, wnv, &groups, &units);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) N += __shfl_xor_sync(kAll, N, o);
  // a block takes four units at least: fewer would leave more to join than they
  // save
  const int64_t G = min((int64_t)gridDim.x, (N + 3) / 4);
  int64_t u = 0, u1 = 0;
  if ((int64_t)blockIdx.x < G) {
    u = N * blockIdx.x / G;
    u1 = N * (blockIdx.x + 1) / G;
  }
  int left = (int)min(u1 - u, (int64_t)INT32_MAX);  // units to come

  // the walk: unit `unit` of segment (b, h, grp); its sequence's numbers
  int b = 0, h = 0, grp = 0, unit = 0, len = 0, nv = 0;
  if (left > 0) {
    int64_t before = 0;
    if (wbase != 0) window(0);
    for (;; window(wbase + 32)) {
      const int64_t mine = att_units<Cfg::kTok>(C.H, wlen, wnv, &groups, &units);
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
        b = wbase + l;
        len = __shfl_sync(kAll, wlen, l);
        nv = __shfl_sync(kAll, wnv, l);
        att_units<Cfg::kTok>(C.H, len, nv, &groups, &units);
        const int64_t hg = at / units;
        unit = (int)(at - hg * units);
        h = (int)(hg / groups);
        grp = (int)(hg - (int64_t)h * groups);
        break;
      }
      before += __shfl_sync(kAll, incl, 31);
    }
  }
  int* rec = A.rec + blockIdx.x * 8;
  if (par == 0 && lane == 0) rec[0] = 0;

  // A batch: the next units of one segment. Lanes NG i .. hold the i-th unit of
  // this warp, lane NG i + s its tokens 16 s ..
  struct Batch {
    int total, n;  // units, and this warp's
    int b, h, q0, rows, len, vis, flags, slot, joins, seg_at;
    int number;    // of this warp's first unit
    int t0, id;    // the lane's unit's first token; the page of its tokens
    float ks, vs;
  };
  const int of = lane / NG, sl = lane % NG;
  // the segment's run in this block: `seg_n` units, `seg_at` of them taken
  int seg_at = 0, seg_n = 0, joins = 0, taken = 0;
  bool seg_whole = false, seg_head = false;

  auto next_batch = [&](Batch& k) {
    k.total = k.n = 0;
    k.id = -1;
    if (left == 0) return;
    const int q0 = grp * kAttRows, rows = min(kAttRows, nv - q0);
    if (seg_at == seg_n) {
      seg_at = 0;
      seg_head = unit == 0;
      seg_n = min(units - unit, left);
      seg_whole = seg_head && seg_n == units;
      if (lane == 0) {
        // by both warps, the same: each orders it before the units it hands out
        if (seg_n > 1) segs[joins % kSegRing] = SegInfo{b, h, q0, rows, seg_whole, seg_head};
        if (par == 0 && seg_head && !seg_whole) {
          // it goes on in the blocks behind: up to which
          const int64_t end = u1 - left + units - 1;
          rec[0] = 1;
          rec[1] = (int)(((end + 1) * G - 1) / N) - (int)blockIdx.x + 1;
          rec[2] = b;
          rec[3] = h;
          rec[4] = q0;
          rec[5] = rows;
        }
      }
    }
    k.total = min(2 * kBatch, seg_n - seg_at);
    const int off = (taken ^ par) & 1;
    k.n = (k.total - off + 1) / 2;
    k.b = b;
    k.h = h;
    k.q0 = q0;
    k.rows = rows;
    k.len = len;
    k.vis = len + q0 + rows;
    k.flags = (seg_n == 1 ? kSolo : 0) | (seg_whole ? kWhole : 0);
    k.slot = seg_head;
    k.joins = joins;
    k.seg_at = seg_at + off;
    k.number = taken + off;
    k.t0 = (unit + off + 2 * of) * Cfg::kTok;
    const int pos = k.t0 + 16 * sl;
    if (of < k.n && pos < k.vis) {
      k.id = page_of(C, S, b, pos >> pshift);
      if (k.id < 0) cache_error(C);
    }
    left -= k.total;
    taken += k.total;
    seg_at += k.total;
    unit += k.total;
    if (seg_at == seg_n && seg_n > 1) ++joins;
    if (unit == units) {
      unit = 0;
      if (++grp == groups) {
        grp = 0;
        if (++h == C.H && left > 0) {
          h = 0;
          do {  // the next sequence with rows
            if (++b == wbase + 32) window(b);
            nv = __shfl_sync(kAll, wnv, b - wbase);
          } while (nv == 0);
          len = __shfl_sync(kAll, wlen, b - wbase);
          att_units<Cfg::kTok>(C.H, len, nv, &groups, &units);
        }
      }
    }
  };
  auto scales = [&](Batch& k) {
    k.ks = k.vs = 0.f;
    if constexpr (I8)
      if (k.id >= 0) {
        const int64_t hs = (int64_t)k.id * C.H + k.h;
        k.ks = C.kscale[hs];
        k.vs = C.vscale[hs];
      }
  };

  int st = par;
  uint32_t ph = 0;
  bool good = true;
  auto next_stage = [&]() {
    if ((st += 2) >= Cfg::kStages) {
      st -= Cfg::kStages;
      ph ^= 1;
    }
  };
  const int chunk = min(C.P / 16, NG);  // groups that lie together in a page
  auto issue = [&](const Batch& k, int i) {
    if (!good || !(good = sm100::mbar_wait(&empty[st], ph ^ 1))) return;
    unsigned char* sp = stages + (size_t)st * Cfg::kStage;
    UnitMeta* mt = reinterpret_cast<UnitMeta*>(sp + Cfg::kMeta);
    const bool mine = of == i;
    const unsigned ok = __ballot_sync(kAll, mine && k.id >= 0);
    const bool first = k.seg_at + 2 * i < kAttWarps;  // a warp's first of the segment
    if (mine) {
      if constexpr (I8) {
        mt->ks[sl] = k.ks;
        mt->vs[sl] = k.vs;
      }
      if (sl == 0) {
        mt->b = k.b;
        mt->h = k.h;
        mt->q0 = k.q0;
        mt->rows = k.rows;
        mt->len = k.len;
        mt->t0 = k.t0;
        mt->vis = k.vis;
        mt->flags = k.flags | (first ? kRows : 0);
        mt->slot = k.slot;
        mt->joins = k.joins;
        mt->n = k.number + 2 * i;
        mt->ok = ok >> (NG * i);
      }
    }
    __syncwarp();
    if (mine && sl == 0)
      sm100::mbar_expect_tx(&full[st],
                            __popc(ok) * (32 * D * Cfg::E + 64) + (first ? k.rows * D * 2 : 0));
    __syncwarp();
    if (mine) {
      if (k.id >= 0) {
        const int pos = k.t0 + 16 * sl, slot = pos & (C.P - 1);
        const int64_t hs = (int64_t)k.id * C.H + k.h;
        const int64_t from = ((hs << pshift) + slot) * (D * Cfg::E);
        if (sl % chunk == 0) {
          const int n = min(chunk, (k.vis - pos + 15) / 16);
          sm100::bulk_copy_g2s(sp + sl * 16 * D * Cfg::E, static_cast<char*>(C.k) + from,
                               n * 16 * D * Cfg::E, &full[st]);
          sm100::bulk_copy_g2s(sp + Cfg::kNorm + sl * 64, C.kinv + (hs << pshift) + slot, n * 64,
                               &full[st]);
        }
        sm100::bulk_copy_g2s(sp + Cfg::kK + sl * Cfg::kVGroup, static_cast<char*>(C.v) + from,
                             16 * D * Cfg::E, &full[st]);
      }
      if (first)
        for (int r = sl; r < k.rows; r += NG)
          sm100::bulk_copy_g2s(sp + Cfg::kX + r * D * 2,
                               A.x + k.b * A.xs[0] + k.h * A.xs[1] + (int64_t)(k.q0 + r) * A.xs[2],
                               D * 2, &full[st]);
    }
    __syncwarp();
    next_stage();
  };

  Batch cur, nxt;
  next_batch(cur);
  scales(cur);
  while (cur.total > 0) {
    // the next batch's page numbers travel while the first half of this batch's
    // copies are issued, its scales behind the second half
    next_batch(nxt);
    const int half = min(cur.n, kBatch / 2);
    for (int i = 0; i < half; ++i) issue(cur, i);
    scales(nxt);
    for (int i = half; i < cur.n; ++i) issue(cur, i);
    cur = nxt;
  }
  for (int i = (taken ^ par) & 1; i < kAttWarps && good; i += 2) {  // an end for every warp
    if (!(good = sm100::mbar_wait(&empty[st], ph ^ 1))) break;
    if (lane == 0) {
      UnitMeta* mt = reinterpret_cast<UnitMeta*>(stages + (size_t)st * Cfg::kStage + Cfg::kMeta);
      mt->flags = kEnd;
      mt->joins = joins;
      mt->n = taken + i;
      sm100::mbar_arrive(&full[st]);
    }
    next_stage();
  }
  if (!good) {
    if (lane == 0 && C.status) record_status(C.status, 5u /* LSH_ERR_TIMEOUT */);
    // let every copy land before the block's memory goes away
    for (int i = 0; i < Cfg::kStages; ++i) {
      sm100::mbar_wait(&full[i], 0, 100000000ull);
      sm100::mbar_wait(&full[i], 1, 100000000ull);
    }
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

__device__ __forceinline__ float att_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool I8>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D, I8>::kBlocks) k_cache_attend(AttendArgs A) {
  using Cfg = AttCfg<D, I8>;
  using T = std::conditional_t<I8, __half, bf16>;
  constexpr int NG = Cfg::kGroups;
  constexpr int kSteps = D / 16;  // 16-wide steps of Q K^T
  constexpr int kN = D / 8;       // 8-wide column tiles of P V
  constexpr int kJ = 2 * NG;      // 8-token tiles of S
  extern __shared__ __align__(16) unsigned char smem[];
  float* merge = reinterpret_cast<float*>(smem);  // [4][8][D]
  float* wm = reinterpret_cast<float*>(smem + Cfg::kMerge);  // [8 warps][8 rows]
  float* wl = wm + 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(wl + 64);
  uint64_t* empty = full + 16;
  SegInfo* segs = reinterpret_cast<SegInfo*>(empty + 16);
  unsigned char* stages = smem + Cfg::kFixed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], 1);
      reinterpret_cast<UnitMeta*>(stages + (size_t)i * Cfg::kStage + Cfg::kMeta)->n = -1;
    }
    sm100::fence_mbar_init();
  }
  __syncthreads();
  if (warp >= kAttWarps) {
    att_copy_warp<D, I8>(A, stages, full, empty, segs, warp - kAttWarps);
    return;
  }
  att_pad_rows<D>(A);

  const float cs = kLog2e / sqrtf((float)D);
  uint32_t qa[2 * kSteps];  // Q as A operand: step s, a0 and a2 (rows g)
  float o[kN][4];
  float m = -INFINITY, l = 0.f, qscale = 1.f;
  float vref = 0.f, vinv = 0.f;  // int8: o counts in units of the scale vref
  // int8: weights are held 2^14 times larger, so that f16 keeps those down to
  // 2^-38 of the largest; l and o are brought back where they leave the loop
  constexpr float kUp = I8 ? 14.f : 0.f, kDown = I8 ? 0x1p-14f : 1.f;
  bool have = false;             // m, l, o are of the segment to join next
  int joined = 0;
  int st = warp % Cfg::kStages;
  uint32_t ph = (warp / Cfg::kStages) & 1;

  // joins segment `joined` over the eight warps
  auto join = [&]() -> bool {
    l += __shfl_xor_sync(~0u, l, 1);
    l += __shfl_xor_sync(~0u, l, 2);
    l *= kDown;
    if (!have) {
      m = -INFINITY;
      l = 0.f;
    }
    if (t == 0) wm[warp * 8 + g] = m;
    if (sm100::bar_sync_any(1, kAttWarps * 32, false)) return false;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, wm[w * 8 + g]);
    float f = ex2(m - (M == -INFINITY ? 0.f : M));  // 0 where the warp has seen nothing
    if (t == 0) wl[warp * 8 + g] = l * f;
    if (I8) f *= vref * kDown;
    float* mine = merge + ((warp & 3) * 8 + g) * D + 2 * t;
    if (warp >= 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        *reinterpret_cast<float2*>(mine + 8 * i) =
            have ? make_float2((o[i][0] + o[i][2]) * f, (o[i][1] + o[i][3]) * f)
                 : make_float2(0.f, 0.f);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (warp < 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float2 e = *reinterpret_cast<float2*>(mine + 8 * i);
        if (have) {
          e.x += (o[i][0] + o[i][2]) * f;
          e.y += (o[i][1] + o[i][3]) * f;
        }
        *reinterpret_cast<float2*>(mine + 8 * i) = e;
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    // a warp takes a row, a lane D / 32 dimensions
    const SegInfo sg = segs[joined % kSegRing];
    if (warp < sg.rows) {
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
      if (sg.whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        alignas(8) bf16 e[DL];
#pragma unroll
        for (int k = 0; k < DL; ++k) e[k] = __float2bfloat16_rn(sum[k] * inv);
        bf16* op = A.out + sg.b * A.os[0] + sg.h * A.os[1] + (int64_t)(sg.q0 + warp) * A.os[2] + lane * DL;
        if constexpr (DL == 4) *reinterpret_cast<uint2*>(op) = *reinterpret_cast<uint2*>(e);
        else *reinterpret_cast<uint32_t*>(op) = *reinterpret_cast<uint32_t*>(e);
        if (lane == 0)
          A.lse[((int64_t)sg.b * A.C.H + sg.h) * A.S.n + sg.q0 + warp] = att_lse(Mr, L);
      } else {
        const int64_t row = ((int64_t)blockIdx.x * 2 + sg.slot) * 8 + warp;
#pragma unroll
        for (int k = 0; k < DL; ++k) A.part[row * D + lane * DL + k] = sum[k];
        if (lane == 0) {
          A.part_ml[row * 2] = Mr;
          A.part_ml[row * 2 + 1] = L;
        }
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");  // the buffers are free
    have = false;
    ++joined;
    return true;
  };

  for (int n = warp;; n += kAttWarps) {
    const unsigned char* sp = stages + (size_t)st * Cfg::kStage;
    const UnitMeta* mt = reinterpret_cast<const UnitMeta*>(sp + Cfg::kMeta);
    if (__any_sync(~0u, !att_wait_unit(mt, &full[st], ph, n))) {
      if (lane == 0 && A.C.status) record_status(A.C.status, 5u /* LSH_ERR_TIMEOUT */);
      sm100::bar_sync_any(1, kAttWarps * 32, true);
      return;
    }
    const int flags = mt->flags;
    while (joined < mt->joins)
      if (!join()) return;
    if (flags & kEnd) break;

    if (flags & kRows) {
      const bool in = g < mt->rows;  // rows that are not there: zeros
      const unsigned char* qp = sp + Cfg::kX + g * D * 2;
      if constexpr (I8) {
        // dimensions 64 j + 16 t .. + 15 of row g: steps 4 j .. 4 j + 3
        float f[D / 4], top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(qp + (64 * (j >> 1) + 16 * t + 8 * (j & 1)) * 2);
          Vec16<bf16>::unpack(in ? u : make_uint4(0, 0, 0, 0), f + 8 * j);
        }
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(f[i]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // a power of two that brings the row's largest value to [1, 2)
        const int e = max(-126, min(126, (int)(__float_as_uint(top) >> 23) - 127));
        qscale = __uint_as_float((uint32_t)(e + 127) << 23);
        const float up = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const __half2 p2 = __floats2half2_rn(f[2 * i] * up, f[2 * i + 1] * up);
          qa[i] = *reinterpret_cast<const uint32_t*>(&p2);
        }
      } else {
        // dimensions 32 j + 8 t .. + 7: steps 2 j and 2 j + 1
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(qp + (32 * j + 8 * t) * 2);
          qa[4 * j] = in ? u.x : 0u;
          qa[4 * j + 1] = in ? u.y : 0u;
          qa[4 * j + 2] = in ? u.z : 0u;
          qa[4 * j + 3] = in ? u.w : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
      m = -INFINITY;
      l = 0.f;
      vref = 0.f;
      have = true;
    }

    // S: column c of tile j is token 2 kJ (c / 2) + 2 j + c % 2, so that this lane
    // holds tokens 2 kJ t .. of row g: tokens 2 j and 2 j + 1 of its own in tile j
    float p[2 * kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const unsigned char* kp = sp + (2 * kJ * (g >> 1) + 2 * j + (g & 1)) * D * Cfg::E + 16 * t;
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
            mma_16816(s, qa[a], 0u, qa[a + 1], 0u, b0, b1, T());
          }
        } else {
          mma_16816(s, qa[4 * i], 0u, qa[4 * i + 1], 0u, u.x, u.y, T());
          mma_16816(s, qa[4 * i + 2], 0u, qa[4 * i + 3], 0u, u.z, u.w, T());
        }
      }
      p[2 * j] = s[0];
      p[2 * j + 1] = s[1];
    }
    const int tok0 = mt->t0 + 2 * kJ * t;  // this lane's first token
    const int grp = 2 * kJ * t / 16;       // and its group
    const uint32_t ok = mt->ok;
    float f = cs;
    if constexpr (I8) f *= mt->ks[grp] * qscale;
#pragma unroll
    for (int j = 0; j < kJ / 2; ++j) {
      const float4 kn = *reinterpret_cast<const float4*>(sp + Cfg::kNorm + (2 * kJ * t + 4 * j) * 4);
      p[4 * j] *= kn.x * f;
      p[4 * j + 1] *= kn.y * f;
      p[4 * j + 2] *= kn.z * f;
      p[4 * j + 3] *= kn.w * f;
    }
    // units with tokens that some row must not see, or that are not there
    const bool tail = mt->t0 + Cfg::kTok > mt->len + mt->q0 || ok != (1u << NG) - 1;
    if (tail) {
      const int self = mt->len + mt->q0 + g - tok0;  // row g's own token
      const bool there = ok >> grp & 1;
#pragma unroll
      for (int k = 0; k < 2 * kJ; ++k)
        p[k] = k > self || !there ? -INFINITY : k == self ? kSelfLogit * kLog2e : p[k];
    }
    float top = p[0];
#pragma unroll
    for (int k = 1; k < 2 * kJ; ++k) top = fmaxf(top, p[k]);
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    const bool up = top > m;
    float corr = up ? ex2(m - top) : 1.f;
    if (up) {
      m = top;
      l *= corr;
    }
    float ratio = 1.f;
    bool again = up;
    if constexpr (I8) {
      // the unit's largest scale: the lanes of a row hold all its groups
      float vs = ok >> grp & 1 ? mt->vs[grp] : 0.f;
      float vm = fmaxf(vs, __shfl_xor_sync(~0u, vs, 1));
      vm = fmaxf(vm, __shfl_xor_sync(~0u, vm, 2));
      if (vm > vref) {
        vinv = 1.f / vm;
        corr *= vref * vinv;
        vref = vm;
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
    const float ref = m == -INFINITY ? 0.f : m - kUp;
#pragma unroll
    for (int k = 0; k < 2 * kJ; ++k) {
      p[k] = ex2(p[k] - ref);
      l += p[k];
      if constexpr (I8) p[k] *= ratio;
    }
    // P as A operand: step s is tiles 2 s and 2 s + 1, high and low part
    uint32_t a[kJ][2];
#pragma unroll
    for (int j = 0; j < kJ; ++j) split2(p[2 * j], p[2 * j + 1], &a[j][0], &a[j][1], T());
    // v: 16 bytes of a dimension are this lane's tokens
    const unsigned char* vp = sp + Cfg::kK + grp * Cfg::kVGroup +
                              (g * 16 + 2 * kJ * t % 16) * Cfg::E;
    if (I8 || !tail) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(vp + i * 128 * Cfg::E);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (I8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1;
            i8_to_f16(w[k], &b0, &b1);
            mma_16816(o[i], a[2 * k][0], a[2 * k][1], a[2 * k + 1][0], a[2 * k + 1][1], b0, b1, T());
          }
        } else {
          mma_16816(o[i], a[0][0], a[0][1], a[1][0], a[1][1], w[0], w[1], T());
          mma_16816(o[i], a[2][0], a[2][1], a[3][0], a[3][1], w[2], w[3], T());
        }
      }
    } else {
      // bf16 values that some row must not see: slots behind the last row, and
      // groups that are not there, hold anything, and a later row's value may be
      // infinite; 0 times it is NaN. The former are cleared; where one of the
      // latter is not finite, the tokens go one by one and each row takes its own.
      const int count = ok >> grp & 1 ? mt->vis - tok0 : 0;  // of this lane's, those there
      uint32_t keep[4], odd = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        keep[k] = count >= 2 * k + 2 ? ~0u : count == 2 * k + 1 ? 0xffffu : 0u;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(vp + i * 256);
        const uint32_t w[4] = {u.x & keep[0], u.y & keep[1], u.z & keep[2], u.w & keep[3]};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          odd |= (uint32_t)((w[k] & 0x7f80u) == 0x7f80u) |
                 (uint32_t)((w[k] & 0x7f800000u) == 0x7f800000u);
        }
      if (!__any_sync(~0u, odd)) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(vp + i * 256);
          mma_16816(o[i], a[0][0], a[0][1], a[1][0], a[1][1], u.x & keep[0], u.y & keep[1], T());
          mma_16816(o[i], a[2][0], a[2][1], a[3][0], a[3][1], u.z & keep[2], u.w & keep[3], T());
        }
      } else {
        for (int tk = 0; tk < Cfg::kTok; ++tk) {
          uint32_t e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            e[k] = tk / (2 * kJ) == t && tk % (2 * kJ) / 2 == k
                       ? keep[k] & (tk & 1 ? 0xffff0000u : 0xffffu)
                       : 0u;
          const bool sees = mt->t0 + tk <= mt->len + mt->q0 + g;
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(vp + i * 256);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_16816(d, a[0][0], a[0][1], a[1][0], a[1][1], u.x & e[0], u.y & e[1], T());
            mma_16816(d, a[2][0], a[2][1], a[3][0], a[3][1], u.z & e[2], u.w & e[3], T());
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (sees) o[i][k] += d[k];
          }
        }
      }
    }

    if (flags & kSolo) {
      // the block's only unit of the segment: no other warp has a part
      l += __shfl_xor_sync(~0u, l, 1);
      l += __shfl_xor_sync(~0u, l, 2);
      l *= kDown;
      if (g < mt->rows) {
        float f1 = I8 ? vref * kDown : 1.f;
        if (flags & kWhole) {
          f1 *= l == 0.f ? 0.f : 1.f / l;
          bf16* op = A.out + mt->b * A.os[0] + mt->h * A.os[1] + (int64_t)(mt->q0 + g) * A.os[2] + 2 * t;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            *reinterpret_cast<__nv_bfloat162*>(op + 8 * i) = __floats2bfloat162_rn(
                (o[i][0] + o[i][2]) * f1, (o[i][1] + o[i][3]) * f1);
          if (t == 0)
            A.lse[((int64_t)mt->b * A.C.H + mt->h) * A.S.n + mt->q0 + g] = att_lse(m, l);
        } else {
          const int64_t row = ((int64_t)blockIdx.x * 2 + mt->slot) * 8 + g;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            *reinterpret_cast<float2*>(A.part + row * D + 8 * i + 2 * t) =
                make_float2((o[i][0] + o[i][2]) * f1, (o[i][1] + o[i][3]) * f1);
          if (t == 0) {
            A.part_ml[row * 2] = m;
            A.part_ml[row * 2 + 1] = l;
          }
        }
      }
      have = false;
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&empty[st]);
    st += kAttWarps;
    while (st >= Cfg::kStages) {
      st -= Cfg::kStages;
      ph ^= 1;
    }
  }
  sm100::bar_sync_any(1, kAttWarps * 32, false);
  // k_cache_combine may be brought in
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
