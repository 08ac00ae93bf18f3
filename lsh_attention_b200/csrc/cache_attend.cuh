// Shared-QK attention of a sequence's newest tokens over the paged cache.
//
// Row t at position p = len + t sees the cached tokens j <= p:
//   l_j = x_t . k_j / (||x_j|| sqrt(d)),  l_p = -1e5,
//   out = sum_j softmax(l)_j v_j,  lse = ln sum_j exp l_j.
// With one row, or a handful, for every sequence and head, each cached byte is
// used once: the kernel is a stream through the cache and is bound by DRAM.
//
// Work. A unit is 8 KB of the cache for one (sequence, head, eight or sixteen
// rows), a segment: 64 tokens (int8, d 64), 32 or 16 (bf16, d 128). Units are numbered
// through sequences, heads, row groups and tokens, and every computing warp of
// the card takes an equal run of them, whatever the lengths are: they are read on
// the device. Warps do not wait for one another. A segment that several of them
// share leaves partial sums in the workspace, which k_cache_combine joins in a
// fixed order.
//
// Block (persistent, one an SM). Four warps copy, each for a quarter of the
// computing warps: four lanes walk a warp's run, look the pages of its next unit
// up and fill its own ring of shared-memory stages by bulk copies.
//
// S = Q K^T and O += P V are warp products (m16n8k16): so few rows do not fill a
// tcgen05 tile, and DRAM allows ten times the tensor work. A contraction's index
// may be permuted at will as long as both operands agree, so a lane takes
// dimensions of K (16 bytes) and tokens of V (four of a group of 16, which lies
// dimension by dimension in the cache) that are consecutive in memory, and feeds
// them to the products as they are: no transposes, no shuffles. Weights go in as
// high and low parts in bf16, 2^-17 together whatever their size, so that P V loses
// nothing against fp32 ones: of eight rows in one product, whose 16 rows hold both,
// of sixteen (calls of more than eight rows) in two.
//
// int8: what bounds the kernel besides DRAM is the instructions that widen the
// bytes. One under a zero (a byte permutation for two) is the bf16 number (q + 128) 2^-133,
// and one multiply-add makes it q / 64, exactly. (Keys fed as f16 subnormals (q + 128) 2^-24,
// the 128 taken off as -128 sum x, need no multiply-add: 83.1 us instead of 83.7 for the 64
// images below. But their sums round at the size of 128 sum |x|, whatever the key's:
// one stored as a few steps of its page's scale, or none, had a logit that was noise.) A
// weight is multiplied by its page's scale before it is split: bf16 has the range for
// it, so that no page's scale costs another page's weights any bits.
//
// Measured (main kernel / with the joining of parts and both launches), of the copy
// rate: one token over 65536, 8 heads of 128, bf16: 48.8 us (0.85) / 53; 64 sequences
// of up to 12288, 8 heads of 64, int8: 78 us (0.81) / 83; five rows of 16 sequences,
// bf16 d 128: 41 / 45. What is left: 3.5 us before the first copy (lengths, the
// place of the run, pages, scales: one load after the other), the joining, and in int8
// 12 us of instructions that DRAM does not hide. Built and slower: eight warps on
// the same 128 tokens with a barrier for each segment (129 us for the int8 case:
// short segments wait); one ring for all warps (its stages change hands, 134);
// one copying warp (194); parts joined by the last of eight neighbours, counted
// with atomics, instead of a second kernel (99: the fences wait for loads under way).
#pragma once

#include "cache.cuh"

namespace lsh {

constexpr float kLog2e = 1.4426950408889634f;

struct AttendArgs {
  CacheView C;
  SeqTables S;
  const bf16* x;
  bf16* out;
  float* lse;
  int64_t xs[3], os[3];
  int groups;      // segments of a (sequence, head), most
  float* part;     // [computing warps][2][rows][D] unnormalised sums of split segments
  float* part_ml;  // [computing warps][2][rows][2] their references (log2) and weights' sums
  int4* rec;       // [B][H][groups]: first warp, how many share it (0: it is whole), rows
};

// A ring stage's header, written by the copying warp and handed over by a barrier of
// its own (`head`): it is read while the unit's tokens still travel.
struct UnitMeta {
  int b, h, q0, rows;   // the segment's first row and how many
  int len, t0;          // tokens before the sequence's rows; the unit's first
  int flags, slot;      // kFirst ...; slot of a partial result
  uint32_t ok;          // bit s: tokens 16 s .. of the unit are there
  float ks[4], vs[4];   // int8: scales of k and v
};
// of the warp's units of a segment: the first, the last, all; nothing follows
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8;

template <int D, bool I8>
struct AttCfg {
  static constexpr int E = I8 ? 1 : 2;
  static constexpr int kTok = 4096 / (D * E);       // tokens of a unit
  static constexpr int kGroups = kTok / 16;
  static constexpr int kV = 4096, kNorm = 8192;     // offsets in a stage
  static constexpr int kMeta = kNorm + kTok * 4;
  static constexpr int kStage = kMeta + 128;
  // computing warps and each one's stages: what registers (128 a thread for d 64,
  // 168 for d 128) and shared memory have room for
  static constexpr int kWarps = D == 64 ? 12 : 8;
  static constexpr int kDepth = D == 64 ? 2 : 3;
  static constexpr int kCopy = 4;                   // copying warps
  static constexpr int kThreads = 32 * (kWarps + kCopy);
  static constexpr int kBars = 768;                 // full, empty and head, 32 each
  static constexpr int kSmem = kBars + kWarps * kDepth * kStage;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four int8 to two pairs of bf16, q / 64: a byte under a zero is the bf16 number
// (q + 128) 2^-133 (its eighth bit is the lowest exponent's); times 2^127, less 2.
// All exact.
__device__ __forceinline__ void i8_to_bf16(uint32_t w, uint32_t* b0, uint32_t* b1) {
  w ^= 0x80808080u;
  const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7f00));   // 2^127
  const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(0xc000));  // -2
  uint32_t lo = __byte_perm(w, 0u, 0x4140), hi = __byte_perm(w, 0u, 0x4342);
  const __nv_bfloat162 a = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&lo), up, off);
  const __nv_bfloat162 b = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&hi), up, off);
  *b0 = *reinterpret_cast<const uint32_t*>(&a);
  *b1 = *reinterpret_cast<const uint32_t*>(&b);
}
// (x, y) as a pair of bf16 and what the pair leaves over, as another.
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const __nv_bfloat162 l =
      __floats2bfloat162_rn(x - __bfloat162float(h.x), y - __bfloat162float(h.y));
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

// A pair of bf16 with what is not finite set to zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const __nv_bfloat162 most = __bfloat162bfloat162(__ushort_as_bfloat16(0x7f7f));
  return w & __hle2_mask(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)), most);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------- the copying warps
// A sequence's row groups and units of a segment of it; all its units.
template <int kTok, int kRows>
__device__ __forceinline__ int64_t att_units(int H, int len, int nv, int* groups, int* units) {
  *groups = (nv + kRows - 1) / kRows;
  *units = (int)(((int64_t)len + nv + kTok - 1) / kTok);
  return (int64_t)H * *groups * *units;
}

// a / b of numbers that are not negative, by 32 bits where they fit.
__device__ __forceinline__ int64_t udiv(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(sm100::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Copying warp `pw`: lanes 4 q .. 4 q + 3 serve computing warp pw kWarps / 4 + q,
// lane 4 q + s the tokens 16 s .. of its units. The lane groups go their own ways.
template <int D, bool I8, int RG>
__device__ void att_copy_warp(const AttendArgs& A, unsigned char* stages, uint64_t* full,
                              uint64_t* empty, uint64_t* head, int pw) {
  using Cfg = AttCfg<D, I8>;
  constexpr int NG = Cfg::kGroups, kServe = Cfg::kWarps / Cfg::kCopy;
  const CacheView& C = A.C;
  const SeqTables& S = A.S;
  const int lane = threadIdx.x & 31, q = lane >> 2, sl = lane & 3;
  const unsigned kAll = 0xffffffffu, mine = 0xfu << (4 * q);
  const int pshift = __ffs(C.P) - 1;
  const int wk = pw * kServe + (q < kServe ? q : 0);  // the computing warp

  // all units; the lanes hold the tokens of 32 sequences
  int wlen = 0, wnv = 0, groups, units;
  auto window = [&](int base) {
    wlen = wnv = 0;
    if (base + lane < S.B) seq_rows(S, C.P, base + lane, &wlen, &wnv);
    return att_units<Cfg::kTok, 8 * RG>(C.H, wlen, wnv, &groups, &units);
  };
  int64_t N = 0, first_window = 0;
  for (int base = 0; base < S.B; base += 32) {
    const int64_t w = window(base);
    if (base == 0) first_window = w;
    N += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) N += __shfl_xor_sync(kAll, N, o);
  // G runs of `each` units, the first `more` of them one longer; neighbouring runs
  // lie in different blocks
  const int64_t G = max((int64_t)1, min((int64_t)gridDim.x * Cfg::kWarps, N));
  const int run = wk * (int)gridDim.x + (int)blockIdx.x;
  const int64_t each = udiv(N, G), more = N - each * G;
  int64_t u = 0;
  int left = 0;  // units to come
  if (q < kServe && run < G) {
    u = run * each + min((int64_t)run, more);
    left = (int)(each + (run < more));
  }
  auto run_of = [&](int64_t x) {  // the run that unit x is in
    return (int)(x < more * (each + 1) ? udiv(x, each + 1) : more + udiv(x - more * (each + 1), each));
  };

  // the walk: unit `unit` of segment (b, h, grp); its sequence's numbers
  int b = 0, h = 0, grp = 0, unit = 0, len = 0, nv = 0;
  groups = units = 1;
  {
    int64_t before = 0;
    bool found = left == 0;
    for (int base = 0; base < S.B && !__all_sync(kAll, found); base += 32) {
      int64_t own = first_window;
      int g0, u0;
      if (S.B > 32) {
        wlen = wnv = 0;
        if (base + lane < S.B) seq_rows(S, C.P, base + lane, &wlen, &wnv);
        own = att_units<Cfg::kTok, 8 * RG>(C.H, wlen, wnv, &g0, &u0);
      }
      int64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += up;
      }
      for (int k = 0; k < kServe; ++k) {
        const int64_t uk = __shfl_sync(kAll, u, 4 * k);
        const unsigned past = __ballot_sync(kAll, before + incl > uk);
        const int l = past ? __ffs(past) - 1 : 0;
        const int64_t at = uk - (before + __shfl_sync(kAll, incl - own, l));
        const int l_len = __shfl_sync(kAll, wlen, l), l_nv = __shfl_sync(kAll, wnv, l);
        if (k == q && past && !found) {
          found = true;
          b = base + l;
          len = l_len;
          nv = l_nv;
          att_units<Cfg::kTok, 8 * RG>(C.H, len, nv, &groups, &units);
          const int64_t hg = udiv(at, units);
          unit = (int)(at - hg * units);
          h = (int)udiv(hg, groups);
          grp = (int)(hg - (int64_t)h * groups);
        }
      }
      before += __shfl_sync(kAll, incl, 31);
    }
  }

  // A unit as it is looked up; `cur` is issued next, its scales under way, `nxt`
  // behind it, its page number under way.
  struct Unit {
    int b, h, q0, rows, len, t0, flags, slot, id;
  };
  Unit cur, nxt;
  float ks = 0.f, vs = 0.f;
  bool begun = false, starts = true;  // the warp has the segment's first unit; a run or segment starts
  auto walk = [&](Unit& k) {
    k.flags = kEnd;
    k.id = -1;
    if (left == 0) return;
    const int q0 = grp * 8 * RG, rows = min(8 * RG, nv - q0);
    if (unit == 0) starts = true;
    if (starts) {
      begun = unit == 0;
      if (begun && sl == 0) {
        int4 r = make_int4(run, 0, rows, 0);
        if (units > left)  // it goes on in the runs behind: up to which
          r.y = run_of(u + units - 1) - run + 1;
        A.rec[((int64_t)b * C.H + h) * A.groups + grp] = r;
      }
    }
    const bool ends = unit == units - 1;
    k.b = b;
    k.h = h;
    k.q0 = q0;
    k.rows = rows;
    k.len = len;
    k.t0 = unit * Cfg::kTok;
    k.flags = (starts ? kFirst : 0) | (ends || left == 1 ? kLast : 0) | (ends && begun ? kWhole : 0);
    k.slot = begun;
    starts = false;
    const int pos = k.t0 + 16 * sl;
    if (sl < NG && pos < len + q0 + rows) {
      k.id = page_of(C, S, b, pos >> pshift);
    }
    --left;
    ++u;
    if (++unit == units) {
      unit = 0;
      if (++grp == groups) {
        grp = 0;
        if (++h == C.H && left > 0) {
          h = 0;
          do {  // the next sequence with rows
            seq_rows(S, C.P, ++b, &len, &nv);
          } while (nv == 0);
          att_units<Cfg::kTok, 8 * RG>(C.H, len, nv, &groups, &units);
        }
      }
    }
  };
  auto scales = [&](const Unit& k) {
    ks = vs = 0.f;
    if constexpr (I8)
      if (k.id >= 0) {
        const int64_t hs = (int64_t)k.id * C.H + k.h;
        ks = C.kscale[hs];
        vs = C.vscale[hs];
      }
  };
  walk(cur);
  walk(nxt);
  scales(cur);

  int st = 0;
  uint32_t ph = 0;
  bool open = q < kServe;  // an end has still to be sent
  const int chunk = min(C.P / 16, NG);  // groups that lie together in a page
  uint64_t t_free = sm100::global_ns();
  while (__any_sync(kAll, open)) {
    const int slot = wk * Cfg::kDepth + st;
    const bool go = __shfl_sync(kAll, open && mbar_test(&empty[slot], ph ^ 1), 4 * q);
    if (!__any_sync(kAll, go)) {
      __nanosleep(32);
      if (sm100::global_ns() - t_free > sm100::kWaitLimitNs) break;
      continue;
    }
    if (go) {
      __syncwarp(mine);  // one lane has seen the stage free, four write to it
      unsigned char* sp = stages + (size_t)slot * Cfg::kStage;
      UnitMeta* mt = reinterpret_cast<UnitMeta*>(sp + Cfg::kMeta);
      const uint32_t ok = (__ballot_sync(mine, cur.id >= 0) >> (4 * q)) & 15;
      if (I8) {
        mt->ks[sl] = ks;
        mt->vs[sl] = vs;
      }
      if (sl == 0) {
        mt->b = cur.b;
        mt->h = cur.h;
        mt->q0 = cur.q0;
        mt->rows = cur.rows;
        mt->len = cur.len;
        mt->t0 = cur.t0;
        mt->flags = cur.flags;
        mt->slot = cur.slot;
        mt->ok = ok;
      }
      __syncwarp(mine);
      if (sl == 0) {
        sm100::mbar_expect_tx(&full[slot], __popc(ok) * (32 * D * Cfg::E + 64));
        sm100::mbar_arrive(&head[slot]);
      }
      __syncwarp(mine);
      if (cur.id >= 0) {
        const int pos = cur.t0 + 16 * sl, ps = pos & (C.P - 1);
        const int64_t hs = (int64_t)cur.id * C.H + cur.h;
        const int64_t from = ((hs << pshift) + ps) * (D * Cfg::E);
        if (sl % chunk == 0) {
          const int take = min(chunk, (cur.len + cur.q0 + cur.rows - pos + 15) / 16);
          sm100::bulk_copy_g2s(sp + sl * 16 * D * Cfg::E, static_cast<char*>(C.k) + from,
                               take * 16 * D * Cfg::E, &full[slot]);
          sm100::bulk_copy_g2s(sp + Cfg::kNorm + sl * 64, C.kinv + (hs << pshift) + ps, take * 64,
                               &full[slot]);
          sm100::bulk_copy_g2s(sp + Cfg::kV + sl * 16 * D * Cfg::E, static_cast<char*>(C.v) + from,
                               take * 16 * D * Cfg::E, &full[slot]);
        }
      } else if (sl < NG && !(cur.flags & kEnd) && cur.t0 + 16 * sl < cur.len + cur.q0 + cur.rows) {
        cache_error(C);  // a bad page
      }
      open = !(cur.flags & kEnd);
      cur = nxt;
      scales(cur);
      walk(nxt);
      if (++st == Cfg::kDepth) {
        st = 0;
        ph ^= 1;
      }
    }
    __syncwarp();
    t_free = sm100::global_ns();
  }
  if (__any_sync(kAll, open)) {
    if (lane == 0 && C.status) record_status(C.status, 5u /* LSH_ERR_TIMEOUT */);
    // let every copy land before the block's memory goes away
    for (int i = lane; i < Cfg::kWarps * Cfg::kDepth; i += 32) {
      sm100::mbar_wait(&full[i], 0, 100000000ull);
      sm100::mbar_wait(&full[i], 1, 100000000ull);
    }
  }
}

// ------------------------------------------------------------- the computing warps
// Rows past a sequence's own are zeros, their lse -inf, and there is nothing to
// join for them; sequences are shared out over the blocks.
template <int D, int kThreads, int kRows>
__device__ void att_pad_rows(const AttendArgs& A) {
  for (int b = blockIdx.x; b < A.S.B; b += gridDim.x) {
    int len, nv;
    if (!seq_rows(A.S, A.C.P, b, &len, &nv) && threadIdx.x == 0) cache_error(A.C);
    const int64_t pad = (int64_t)(A.S.n - nv) * A.C.H;
    for (int64_t i = threadIdx.x; i < pad * (D / 8); i += kThreads) {
      const int64_t r = i / (D / 8);
      const int h = (int)(r % A.C.H), t = nv + (int)(r / A.C.H);
      *reinterpret_cast<uint4*>(A.out + b * A.os[0] + h * A.os[1] + t * A.os[2] +
                                i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
      if (i % (D / 8) == 0) A.lse[((int64_t)b * A.C.H + h) * A.S.n + t] = -INFINITY;
    }
    const int full = (nv + kRows - 1) / kRows, none = A.groups - full;
    for (int64_t i = threadIdx.x; i < (int64_t)none * A.C.H; i += kThreads)
      A.rec[((int64_t)b * A.C.H + i / none) * A.groups + full + i % none] = make_int4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ float att_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// RG: rows of a segment, in eights.
template <int D, bool I8, int RG>
__global__ void __launch_bounds__(AttCfg<D, I8>::kThreads, 1) k_cache_attend(AttendArgs A) {
  using Cfg = AttCfg<D, I8>;
  constexpr int NG = Cfg::kGroups;
  constexpr int kSteps = D / 16;  // 16-wide steps of Q K^T
  constexpr int kN = D / 8;       // 8-wide column tiles of P V
  extern __shared__ __align__(16) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + 32;
  uint64_t* head = full + 64;
  unsigned char* stages = smem + Cfg::kBars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  // k_cache_combine may be brought in where there is room: it waits for our end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x < Cfg::kWarps * Cfg::kDepth) {
    sm100::mbar_init(&full[threadIdx.x], 1);
    sm100::mbar_init(&empty[threadIdx.x], 1);
    sm100::mbar_init(&head[threadIdx.x], 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  if (warp >= Cfg::kWarps) {
    att_copy_warp<D, I8, RG>(A, stages, full, empty, head, warp - Cfg::kWarps);
    return;
  }
  att_pad_rows<D, Cfg::kWarps * 32, 8 * RG>(A);

  constexpr float kOver = 7.f;  // a row's reference is moved when a logit passes it by that
  const float cs = kLog2e / sqrtf((float)D);
  // this lane's rows: g and, of sixteen, g + 8
  uint32_t qa[RG][2 * kSteps];  // Q as A operand: step s, a0 and a2 (a1 and a3)
  float o[kN][4];               // eight rows: low parts' sums in the second half
                                // (int8: in units of 64 vref)
  float m[RG], l[RG];           // a row's reference; sum of this lane's weights
  // int8: a power of two, a scale of v that was met, and 1 / vref. It is moved only by
  // a scale 2^64 times larger: its purpose is the range alone, any ratio is exact
  float vref = 0.f, vinv = 0.f;
  int st = 0;
  uint32_t ph = 0;

  for (;;) {
    const int slot = warp * Cfg::kDepth + st;
    const unsigned char* sp = stages + (size_t)slot * Cfg::kStage;
    const UnitMeta* mt = reinterpret_cast<const UnitMeta*>(sp + Cfg::kMeta);
    // the header is there once the unit is issued: a new segment's rows are
    // fetched while its first tokens travel
    if (__any_sync(~0u, !sm100::mbar_wait(&head[slot], ph))) break;
    const int flags = mt->flags;
    if (flags & kEnd) break;
    if (flags & kFirst) {
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const int row = g + 8 * r;
        const bool in = row < mt->rows;  // rows that are not there: zeros
        const bf16* qp =
            A.x + mt->b * A.xs[0] + mt->h * A.xs[1] + (int64_t)(mt->q0 + (in ? row : 0)) * A.xs[2];
        uint4 raw[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          // int8: dimensions 64 j + 16 t .. + 15 are steps 4 j .. 4 j + 3; bf16:
          // dimensions 32 j + 8 t .. + 7 are steps 2 j and 2 j + 1
          raw[j] = *reinterpret_cast<const uint4*>(
              qp + (I8 ? 64 * (j >> 1) + 16 * t + 8 * (j & 1) : 32 * j + 8 * t));
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          if (!in) raw[j] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          qa[r][4 * j] = raw[j].x;
          qa[r][4 * j + 1] = raw[j].y;
          qa[r][4 * j + 2] = raw[j].z;
          qa[r][4 * j + 3] = raw[j].w;
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
      vref = vinv = 0.f;
    }
    if (__any_sync(~0u, !sm100::mbar_wait(&full[slot], ph))) break;

    // S, two tiles of eight tokens for each group of 16: column c of tile e is the
    // group's token 4 (c / 2) + 2 e + c % 2, so that this lane holds its tokens
    // 4 t .. 4 t + 3 for its rows
    float p[RG][NG][4];
    auto q_of = [&](int r, int i) { return r < RG ? qa[r % RG][i] : 0u; };
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const unsigned char* kp = sp + (16 * j + 4 * (g >> 1) + 2 * e + (g & 1)) * D * Cfg::E + 16 * t;
#pragma unroll
        for (int i = 0; i < D * Cfg::E / 64; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(kp + 64 * i);
          if constexpr (I8) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t b0, b1;
              i8_to_bf16(w[k], &b0, &b1);
              const int a = 2 * (4 * i + k);
              mma_16816(s, q_of(0, a), q_of(1, a), q_of(0, a + 1), q_of(1, a + 1), b0, b1);
            }
          } else {
            mma_16816(s, q_of(0, 4 * i), q_of(1, 4 * i), q_of(0, 4 * i + 1), q_of(1, 4 * i + 1), u.x,
                      u.y);
            mma_16816(s, q_of(0, 4 * i + 2), q_of(1, 4 * i + 2), q_of(0, 4 * i + 3),
                      q_of(1, 4 * i + 3), u.z, u.w);
          }
        }
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          p[r][j][2 * e] = s[2 * r];
          p[r][j][2 * e + 1] = s[2 * r + 1];
        }
      }
    const uint32_t ok = mt->ok;
    const int row0 = mt->len + mt->q0;  // position of row 0
    float vtop = 0.f;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const float4 kn = *reinterpret_cast<const float4*>(sp + Cfg::kNorm + (16 * j + 4 * t) * 4);
      if constexpr (I8) vtop = fmaxf(vtop, mt->vs[j]);
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        // (int8: the product with the key as it stands first: 1/||x_j|| times the scale may
        // overflow where the key is stored as zeros)
        const float f = I8 ? cs * 64.f * mt->ks[j] : cs;
        p[r][j][0] = I8 ? p[r][j][0] * f * kn.x : p[r][j][0] * (kn.x * f);
        p[r][j][1] = I8 ? p[r][j][1] * f * kn.y : p[r][j][1] * (kn.y * f);
        p[r][j][2] = I8 ? p[r][j][2] * f * kn.z : p[r][j][2] * (kn.z * f);
        p[r][j][3] = I8 ? p[r][j][3] * f * kn.w : p[r][j][3] * (kn.w * f);
      }
    }
    // units with tokens that some row must not see, or that are not there
    const bool tail = mt->t0 + Cfg::kTok > row0 || ok != (1u << NG) - 1;
    if (tail) {
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const int self = row0 + g + 8 * r - (mt->t0 + 16 * j + 4 * t);  // the row's own token
          const bool there = ok >> j & 1;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            p[r][j][k] = k > self || !there ? -INFINITY : k == self ? kSelfLogit * kLog2e : p[r][j][k];
        }
    }
    float top[RG];
    const bool vover = I8 && vtop > vref * 0x1p64f;
    bool over = vover;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      top[r] = -INFINITY;
#pragma unroll
      for (int j = 0; j < NG; ++j)
        top[r] = fmaxf(top[r], fmaxf(fmaxf(p[r][j][0], p[r][j][1]), fmaxf(p[r][j][2], p[r][j][3])));
      over |= top[r] > m[r] + kOver;
    }
    if (__any_sync(~0u, over)) {
      float corr[RG], down = 1.f;
      if (vover) {
        const float was = vref;
        vref = __uint_as_float(min(max(__float_as_uint(vtop) & 0x7f800000u, 0x00800000u), 0x7e800000u));
        vinv = recip2(vref);
        down = was * vinv;
      }
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
        corr[r] = 1.f;
        if (top[r] > m[r]) {
          corr[r] = ex2(m[r] - top[r]);
          m[r] = top[r];
          l[r] *= corr[r];
        }
        if (I8) corr[r] *= down;
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= corr[RG == 2 ? k >> 1 : 0];
    }
    // P as A operand: the step of group j is its two tiles; high and low part
    uint32_t a[RG][NG][2], al[RG][NG][2];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      // int8: weights of V carry their group's scale
      const float vs = I8 ? mt->vs[j] * vinv : 1.f;
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float ref = m[r] == -INFINITY ? 0.f : m[r];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[r][j][k] = ex2(p[r][j][k] - ref);
          sum += p[r][j][k];
          if (I8) p[r][j][k] *= vs;
        }
        l[r] += sum;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          split2(p[r][j][2 * e], p[r][j][2 * e + 1], &a[r][j][e], &al[r][j][e]);
      }
    }
    // d += P V of group j's tokens for one tile of dimensions. An infinite or NaN
    // value counts with the weights' high parts alone: low ones are zeros or of either sign
    auto product = [&](float (&d)[4], int j, uint32_t b0, uint32_t b1) {
      if constexpr (RG == 1) {
        mma_16816(d, a[0][j][0], al[0][j][0], a[0][j][1], al[0][j][1], b0, b1);
      } else {
        mma_16816(d, a[0][j][0], a[RG - 1][j][0], a[0][j][1], a[RG - 1][j][1], b0, b1);
        mma_16816(d, al[0][j][0], al[RG - 1][j][0], al[0][j][1], al[RG - 1][j][1],
                  I8 ? b0 : finite2(b0), I8 ? b1 : finite2(b1));
      }
    };
    // v: four tokens of a dimension, 4 or 8 bytes
    const unsigned char* vp = sp + Cfg::kV + (g * 16 + 4 * t) * Cfg::E;
    auto load_v = [&](int j, int i, uint32_t* b0, uint32_t* b1) {
      const unsigned char* at = vp + j * 16 * D * Cfg::E + i * 128 * Cfg::E;
      if constexpr (I8) {
        i8_to_bf16(*reinterpret_cast<const uint32_t*>(at), b0, b1);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(at);
        *b0 = u.x;
        *b1 = u.y;
      }
    };
    if (I8 || !tail) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          uint32_t b0, b1;
          load_v(j, i, &b0, &b1);
          product(o[i], j, b0, b1);
        }
    } else if constexpr (!I8) {
      // bf16 values that some row must not see: slots behind the last row, and
      // groups that are not there, hold anything, and a later row's value may be
      // infinite; 0 times it is NaN. The former are cleared; where one of the
      // latter is not finite, the tokens go one by one and each row takes its own.
      uint32_t k0[NG], k1[NG], odd = 0;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        // of this lane's tokens, those that count
        const int count = ok >> j & 1 ? row0 + mt->rows - (mt->t0 + 16 * j + 4 * t) : 0;
        k0[j] = count >= 2 ? ~0u : count == 1 ? 0xffffu : 0u;
        k1[j] = count >= 4 ? ~0u : count == 3 ? 0xffffu : 0u;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          uint32_t b0, b1;
          load_v(j, i, &b0, &b1);
          b0 &= k0[j];
          b1 &= k1[j];
          odd |= (uint32_t)((b0 & 0x7f80u) == 0x7f80u) | (uint32_t)((b0 & 0x7f800000u) == 0x7f800000u) |
                 (uint32_t)((b1 & 0x7f80u) == 0x7f80u) | (uint32_t)((b1 & 0x7f800000u) == 0x7f800000u);
        }
      }
      const bool apart = __any_sync(~0u, odd);
      for (int tk = 0; tk < (apart ? Cfg::kTok : 1); ++tk) {
        bool sees[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) sees[r] = !apart || mt->t0 + tk <= row0 + g + 8 * r;
        const uint32_t half = tk & 1 ? 0xffff0000u : 0xffffu;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            uint32_t b0, b1;
            load_v(j, i, &b0, &b1);
            const bool here = tk / 16 == j && tk % 16 / 4 == t;
            b0 &= !apart ? k0[j] : here && !(tk & 2) ? half & k0[j] : 0u;
            b1 &= !apart ? k1[j] : here && (tk & 2) ? half & k1[j] : 0u;
            product(d, j, b0, b1);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (sees[RG == 2 ? k >> 1 : 0]) o[i][k] += d[k];
        }
      }
    }

    if (flags & kLast) {
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        float L = l[r] + __shfl_xor_sync(~0u, l[r], 1);
        L += __shfl_xor_sync(~0u, L, 2);
        const int row = g + 8 * r;
        if (row >= mt->rows) continue;
        float f = I8 ? 64.f : 1.f;
        const float unit = I8 ? vref : 1.f;
        if (flags & kWhole) f *= L == 0.f ? 0.f : 1.f / L;
        auto value = [&](int i, int k) {
          float y = o[i][2 * r + k];
          if (RG == 1 && fabsf(y) < INFINITY) y += o[i][2 + k];  // (low parts, as in product)
          return y * f * unit;
        };
        if (flags & kWhole) {
          bf16* op = A.out + mt->b * A.os[0] + mt->h * A.os[1] + (int64_t)(mt->q0 + row) * A.os[2] + 2 * t;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            *reinterpret_cast<__nv_bfloat162*>(op + 8 * i) =
                __floats2bfloat162_rn(value(i, 0), value(i, 1));
          if (t == 0)
            A.lse[((int64_t)mt->b * A.C.H + mt->h) * A.S.n + mt->q0 + row] = att_lse(m[r], L);
        } else {
          const int64_t run = (int64_t)warp * gridDim.x + blockIdx.x;
          const int64_t at = (run * 2 + mt->slot) * 8 * RG + row;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            *reinterpret_cast<float2*>(A.part + at * D + 8 * i + 2 * t) =
                make_float2(value(i, 0), value(i, 1));
          if (t == 0) *reinterpret_cast<float2*>(A.part_ml + at * 2) = make_float2(m[r], L);
        }
      }
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&empty[slot]);
    if (++st == Cfg::kDepth) {
      st = 0;
      ph ^= 1;
    }
  }
  // (a wait that gave up is recorded by the copying warp, which gives up as well)
}

// Joins the parts of a row that several warps of k_cache_attend have left: the
// first one's last, then the first of each behind it. A row's 32 dimensions a
// block, eight lanes for a part, so that all parts' loads are under way at once:
// the time is that of two loads from L2 in turn and the launch. The order in
// which parts are summed is that of their numbers.
// grid (segments, up to kRows rows, D / 32), block 8 x parts or so, 32 .. 256.
template <int D, int kRows>
__global__ void __launch_bounds__(256) k_cache_combine(AttendArgs A) {
  constexpr int kAt = 5;  // parts of a lane that are fetched together
  const int lane8 = threadIdx.x & 7, ps = threadIdx.x >> 3, slots = blockDim.x >> 3;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = blockIdx.x, row = blockIdx.y, dim0 = blockIdx.z * 32;
  __shared__ float sm[8], sl[8];
  __shared__ __align__(16) float so[8][32];
  // launched while k_cache_attend still runs: wait for its end, and its writes
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 r = A.rec[seg];
  const int count = r.y;
  if (count == 0 || row >= r.z) return;
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = ps; j0 < count; j0 += kAt * slots) {
    float2 ml[kAt];
    float4 pv[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int j = j0 + i * slots;
      ml[i] = make_float2(-INFINITY, 0.f);
      pv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < count) {
        const int64_t at = (((int64_t)r.x + j) * 2 + (j == 0)) * kRows + row;
        ml[i] = *reinterpret_cast<const float2*>(A.part_ml + at * 2);
        pv[i] = *reinterpret_cast<const float4*>(A.part + at * D + dim0 + lane8 * 4);
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kAt; ++i) top = fmaxf(top, ml[i].x);
    const float ref = top == -INFINITY ? 0.f : top, was = ex2(M - ref);
    L *= was;
    o.x *= was;
    o.y *= was;
    o.z *= was;
    o.w *= was;
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const float f = ex2(ml[i].x - ref);
      L = fmaf(ml[i].y, f, L);
      o.x = fmaf(pv[i].x, f, o.x);
      o.y = fmaf(pv[i].y, f, o.y);
      o.z = fmaf(pv[i].z, f, o.z);
      o.w = fmaf(pv[i].w, f, o.w);
    }
    M = top;
  }
#pragma unroll
  for (int off = 8; off < 32; off <<= 1) {
    const float M2 = __shfl_xor_sync(~0u, M, off), L2 = __shfl_xor_sync(~0u, L, off);
    const float4 o2 = make_float4(__shfl_xor_sync(~0u, o.x, off), __shfl_xor_sync(~0u, o.y, off),
                                  __shfl_xor_sync(~0u, o.z, off), __shfl_xor_sync(~0u, o.w, off));
    const float top = fmaxf(M, M2), ref = top == -INFINITY ? 0.f : top;
    const float f = ex2(M - ref), f2 = ex2(M2 - ref);
    L = L * f + L2 * f2;
    o.x = o.x * f + o2.x * f2;
    o.y = o.y * f + o2.y * f2;
    o.z = o.z * f + o2.z * f2;
    o.w = o.w * f + o2.w * f2;
    M = top;
  }
  if (lane < 8) *reinterpret_cast<float4*>(&so[warp][4 * lane]) = o;
  if (lane == 0) {
    sm[warp] = M;
    sl[warp] = L;
  }
  __syncthreads();
  if (warp != 0) return;
  const int warps = blockDim.x >> 5;
  for (int w = 1; w < warps; ++w) M = fmaxf(M, sm[w]);
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  L = 0.f;
  for (int w = 0; w < warps; ++w) {
    const float f = ex2(sm[w] - ref);
    L += sl[w] * f;
    sum += so[w][lane] * f;
  }
  const int grp = seg % A.groups, bh = seg / A.groups, t = grp * kRows + row;
  const int b = bh / A.C.H, h = bh - b * A.C.H;
  A.out[b * A.os[0] + h * A.os[1] + (int64_t)t * A.os[2] + dim0 + lane] =
      __float2bfloat16_rn(L == 0.f ? 0.f : sum / L);
  if (lane == 0 && dim0 == 0) A.lse[((int64_t)b * A.C.H + h) * A.S.n + t] = att_lse(M, L);
}

}  // namespace lsh
