// The paged cache: what its kernels share, and the kernels that write rows into
// it and read them back.
#pragma once

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

// Smallest power of two s >= 2^-126 with amax <= 127 s. amax finite, >= 0.
__device__ __forceinline__ float scale_for(float amax) {
  int e;
  const float m = frexpf(amax, &e);  // amax = m 2^e, m in [0.5, 1) or 0
  e = m == 0.f ? -126 : e - 7 + (m > 127.f / 128.f);
  return ldexpf(1.f, max(e, -126));
}

// x / s rounded to the nearest integer (ties to even) in [-127, 127]; NaN to 0.
// rs = 1 / s, a power of two, so the product is exact.
__device__ __forceinline__ int quant(float x, float rs) {
  const float q = fminf(fmaxf(rintf(x * rs), -127.f), 127.f);
  return x == x ? (int)q : 0;
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
  int rows;       // tokens a block covers (aligned in the sequence): a multiple
                  // of 16; int8: the page
  int heads_per;  // heads a block takes one after the other
};

inline size_t append_smem(int rows, int d, int pairs) {
  return (size_t)rows * (2 * (d * 2 + 16) + pairs * 8) + 64 * sizeof(float);
}

// Turn the rows [r0, r1) of `xt` in place, W pairs at a time.
template <int D, int W, bool ADJ>
__device__ __forceinline__ void append_rotate(const RotPlan& R, bf16* xt, const float* ct,
                                              const float* st, int r0, int r1) {
  constexpr int kSlots = D / (2 * W);
  for (int i = threadIdx.x; i < (r1 - r0) * kSlots; i += blockDim.x) {
    const int r = r0 + i / kSlots;
    int ra, rb, p;
    rot_slot<W, ADJ>(R, i % kSlots, &ra, &rb, &p);
    if (p >= R.pairs) continue;
    bf16* row = xt + r * (D + 8);
    float u[W], w[W], c[W], s[W];
    Pack<bf16, W>::load(row + ra, u);
    Pack<bf16, W>::load(row + rb, w);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const bool in = p + k < R.pairs;
      c[k] = in ? ct[r * R.pairs + p + k] : 1.f;
      s[k] = in ? st[r * R.pairs + p + k] : 0.f;
    }
    rot_apply<W, ADJ>(u, w, c, s, R.pairs - p);
    Pack<bf16, W>::store(row + ra, u);
    Pack<bf16, W>::store(row + rb, w);
  }
}

// One block: `rows` consecutive token slots of one sequence (int8: one page) for
// a few heads. The sines of its tokens are formed once and serve its heads. Per
// head: rows of x and v into shared memory (cp.async), 1/||x||, rotation in
// place, the rotated rows out by 16-byte pieces; v leaves through transposed
// 8x8 tiles (ldmatrix) so that each thread stores four tokens of a dimension
// together. int8 adds the largest magnitudes over the page in between; this
// block alone owns the page's head, so an earlier row is re-rounded in place.
// W: pairs a thread turns together, 0 = none.
// grid (blocks of rows, head groups, batch), block 256.
template <int D, bool I8, int W, bool ADJ>
__global__ void __launch_bounds__(256) k_cache_append(AppendArgs A) {
  constexpr int kStride = D + 8;  // elements of a shared row: 16 bytes of padding
  constexpr int kPieces = D / 8;  // 16-byte pieces of a row
  const CacheView& C = A.C;
  const int b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = A.S.n, R = A.rows;
  const int h0 = blockIdx.y * A.heads_per, h1 = min(h0 + A.heads_per, C.H);
  int len, nv;
  if (!seq_rows(A.S, C.P, b, &len, &nv) && blockIdx.x == 0 && tid == 0) cache_error(C);

  // rows of xr past the sequence's own: zeros
  if (A.xr) {
    const int t0 = max(nv, (int)min((int64_t)T, (int64_t)blockIdx.x * R));
    const int t1 = (int)min((int64_t)T, (int64_t)(blockIdx.x + 1) * R);
    const int pad = max(t1 - t0, 0) * (h1 - h0) * kPieces;
    for (int i = tid; i < pad; i += 256) {
      const int piece = i % kPieces, rest = i / kPieces;
      const int h = h0 + rest % (h1 - h0), t = t0 + rest / (h1 - h0);
      *reinterpret_cast<uint4*>(A.xr + b * A.os[0] + h * A.os[1] + t * A.os[2] + piece * 8) =
          make_uint4(0, 0, 0, 0);
    }
  }

  // the block's slots: positions base .. base + R - 1; new rows [r0, r1) of them
  const int64_t base = (int64_t)(len / R + blockIdx.x) * R;
  const int r0 = (int)max((int64_t)0, len - base);
  const int r1 = (int)max((int64_t)0, min((int64_t)R, (int64_t)len + nv - base));
  if (r0 >= r1) return;
  const int tok0 = (int)(base - len);  // row r is the call's row tok0 + r

  extern __shared__ __align__(16) unsigned char smem[];
  bf16* xt = reinterpret_cast<bf16*>(smem);
  bf16* vt = xt + R * kStride;
  float* ct = reinterpret_cast<float*>(vt + R * kStride);
  float* st = ct + R * A.rot.pairs;
  float* red = st + R * A.rot.pairs;  // 2 x 8 maxima, then 2 scales old and new

  if constexpr (W > 0) {
    const int pairs = A.rot.pairs;
    for (int i = tid; i < (r1 - r0) * pairs; i += 256) {
      const int r = r0 + i / pairs, p = i % pairs;
      const int ax = rot_axis(A.rot, p);
      rot_angle(A.pos[ax * A.pos_axis + b * A.pos_batch + tok0 + r], A.freqs[p],
                &ct[r * pairs + p], &st[r * pairs + p]);
    }
  }
  // bad pages: rows of xr are still written, the cache is not
  for (int r = r0 + tid; r < r1; r += 256)
    if ((r == r0 || (base + r) % C.P == 0) && page_of(C, A.S, b, (int)((base + r) / C.P)) < 0)
      cache_error(C);

  for (int h = h0; h < h1; ++h) {
    const int own = (r1 - r0) * kPieces;  // pieces of the new rows
    for (int i = tid; i < own; i += 256) {
      const int r = r0 + i / kPieces, piece = i % kPieces;
      const int64_t t = tok0 + r;
      sm100::cp_async16_zfill(xt + r * kStride + piece * 8,
                              A.x + b * A.xs[0] + h * A.xs[1] + t * A.xs[2] + piece * 8, true);
      sm100::cp_async16_zfill(vt + r * kStride + piece * 8,
                              A.v + b * A.vs[0] + h * A.vs[1] + t * A.vs[2] + piece * 8, true);
    }
    sm100::cp_async_commit();
    sm100::cp_async_wait_all();

    // 1/||x|| from the pieces this thread has copied: the row scaled by a power
    // of two near its largest value, so that no square is lost
    for (int i0 = 0; i0 < own; i0 += 256) {
      const int i = i0 + tid;
      const bool in = i < own;
      const int r = r0 + i / kPieces, piece = i % kPieces;
      float f[8];
      if (in) Pack<bf16, 8>::load(xt + r * kStride + piece * 8, f);
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = in ? fmaxf(m, fabsf(f[k])) : 0.f;
#pragma unroll
      for (int o = kPieces / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      int e;
      frexpf(m, &e);
      e = m > 0.f && m <= 3.4e38f ? max(min(e, 126), -126) : 0;
      const float up = ldexpf(1.f, -e);
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = in ? fmaf(f[k] * up, f[k] * up, ss) : 0.f;
#pragma unroll
      for (int o = kPieces / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
      if (in && piece == 0) {
        const int id = page_of(C, A.S, b, (int)((base + r) / C.P));
        const float norm = sqrtf(ss) * ldexpf(1.f, e);
        if (id >= 0)
          C.kinv[((int64_t)id * C.H + h) * C.P + (base + r) % C.P] =
              norm < 1.17549435e-38f ? 0.f : 1.f / norm;
      }
    }
    __syncthreads();
    if constexpr (W > 0) {
      append_rotate<D, W, ADJ>(A.rot, xt, ct, st, r0, r1);
      __syncthreads();
    }

    // the rotated rows: out, and into the cache (bf16)
    float kmax = 0.f, vmax = 0.f;
    bool odd = false;
    for (int i = tid; i < own; i += 256) {
      const int r = r0 + i / kPieces, piece = i % kPieces;
      const uint4 u = *reinterpret_cast<const uint4*>(xt + r * kStride + piece * 8);
      if (A.xr)
        *reinterpret_cast<uint4*>(A.xr + b * A.os[0] + h * A.os[1] +
                                  (int64_t)(tok0 + r) * A.os[2] + piece * 8) = u;
      if constexpr (I8) {
        float f[8], g[8];
        Vec16<bf16>::unpack(u, f);
        Pack<bf16, 8>::load(vt + r * kStride + piece * 8, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool fk = fabsf(f[k]) <= 3.4e38f, gk = fabsf(g[k]) <= 3.4e38f;
          if (fk) kmax = fmaxf(kmax, fabsf(f[k]));
          if (gk) vmax = fmaxf(vmax, fabsf(g[k]));
          odd |= !fk || !gk;
        }
      } else {
        const int id = page_of(C, A.S, b, (int)((base + r) / C.P));
        if (id >= 0)
          *reinterpret_cast<uint4*>(static_cast<bf16*>(C.k) + page_base(C, id, h) +
                                    (base + r) % C.P * D + piece * 8) = u;
      }
    }

    if constexpr (!I8) {
      // v: warps take the block's groups of 16 tokens, 32 dimensions a step
      const int g0 = r0 / kGroup, g1 = (r1 - 1) / kGroup;
      constexpr int kSteps = D / 16;
      for (int w = warp; w < (g1 - g0 + 1) * kSteps; w += 8) {
        const int grp = g0 + w / kSteps, dim0 = (w % kSteps) * 16;
        const int rb = grp * kGroup;
        // tiles 0, 1: tokens {0,1,4,5,8,9,12,13} and {2,3,6,7,10,11,14,15} of
        // dimensions dim0..; tiles 2, 3 the same of the next eight: lane (g, t)
        // then holds tokens 4t .. 4t + 3 of dimensions dim0 + g and dim0 + 8 + g
        const int i = lane & 7, tile = lane >> 3;
        const int trow = rb + (i >> 1) * 4 + (i & 1) + 2 * (tile & 1);
        uint32_t m[4];
        ldsm_x4_trans(m, vt + trow * kStride + dim0 + 8 * (tile >> 1));
        const int64_t at = base + rb;
        const int id = page_of(C, A.S, b, (int)(at / C.P));
        if (id < 0) continue;
        bf16* dst = static_cast<bf16*>(C.v) + page_base(C, id, h) +
                    at % C.P * D + (dim0 + (lane >> 2)) * kGroup + (lane & 3) * 4;
        const int tk = rb + (lane & 3) * 4;
#pragma unroll
        for (int k = 0; k < 2; ++k, dst += 8 * kGroup) {
          if (tk >= r0 && tk + 4 <= r1) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(m[2 * k], m[2 * k + 1]);
          } else {
            uint16_t* e = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (tk + q >= r0 && tk + q < r1)
                e[q] = (uint16_t)(m[2 * k + (q >> 1)] >> (16 * (q & 1)));
          }
        }
      }
    } else {
      if (__syncthreads_or(odd) && tid == 0) cache_error(C);
      kmax = warp_max(kmax);
      vmax = warp_max(vmax);
      if (lane == 0) {
        red[warp] = kmax;
        red[8 + warp] = vmax;
      }
      __syncthreads();
      const int id = page_of(C, A.S, b, (int)(base / C.P));
      if (id >= 0) {
        const int64_t hs = (int64_t)id * C.H + h;
        if (tid < 2) {
          float m = 0.f;
          for (int k = 0; k < 8; ++k) m = fmaxf(m, red[8 * tid + k]);
          float* sc = tid ? C.vscale : C.kscale;
          const float was = r0 > 0 ? sc[hs] : 0.f;
          const float now = fmaxf(was, scale_for(m));
          if (now != was) sc[hs] = now;
          red[16 + 2 * tid] = was;
          red[17 + 2 * tid] = now;
        }
      }
      __syncthreads();
      if (id >= 0) {
        const float kwas = red[16], know = red[17], vwas = red[18], vnow = red[19];
        int8_t* kp = static_cast<int8_t*>(C.k) + page_base(C, id, h);
        int8_t* vp = static_cast<int8_t*>(C.v) + page_base(C, id, h);
        const float krs = 1.f / know, vrs = 1.f / vnow;
        // earlier rows of the page at the raised scale (the ratio is a power of two)
        if (r0 > 0 && know != kwas) {
          const float f = kwas * krs;
          for (int i = tid; i < r0 * D / 4; i += 256) {
            char4 q = *reinterpret_cast<char4*>(kp + 4 * i);
            q.x = (signed char)rintf(q.x * f);
            q.y = (signed char)rintf(q.y * f);
            q.z = (signed char)rintf(q.z * f);
            q.w = (signed char)rintf(q.w * f);
            *reinterpret_cast<char4*>(kp + 4 * i) = q;
          }
        }
        for (int i = tid; i < own; i += 256) {
          const int r = r0 + i / kPieces, piece = i % kPieces;
          float f[8];
          Pack<bf16, 8>::load(xt + r * kStride + piece * 8, f);
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k >> 2] |= (uint32_t)(quant(f[k], krs) & 255) << (8 * (k & 3));
          *reinterpret_cast<uint2*>(kp + r * D + piece * 8) = make_uint2(w[0], w[1]);
        }
        const bool again = r0 > 0 && vnow != vwas;
        const float vf = vwas * vrs;
        const int g0 = again ? 0 : r0 / kGroup, g1 = (r1 - 1) / kGroup;
        constexpr int kSteps = D / 16;
        for (int w = warp; w < (g1 - g0 + 1) * kSteps; w += 8) {
          const int grp = g0 + w / kSteps, dim0 = (w % kSteps) * 16;
          const int rb = grp * kGroup;
          const int i = lane & 7, tile = lane >> 3;
          const int trow = rb + (i >> 1) * 4 + (i & 1) + 2 * (tile & 1);
          uint32_t m[4];
          ldsm_x4_trans(m, vt + trow * kStride + dim0 + 8 * (tile >> 1));
          int8_t* dst = vp + rb * D + (dim0 + (lane >> 2)) * kGroup + (lane & 3) * 4;
          const int tk = rb + (lane & 3) * 4;
#pragma unroll
          for (int k = 0; k < 2; ++k, dst += 8 * kGroup) {
            if (tk >= r1 || (tk + 4 <= r0 && !again)) continue;
            char4 q = make_char4(0, 0, 0, 0);
            if (tk < r0 || tk + 4 > r1) q = *reinterpret_cast<char4*>(dst);
            signed char* e = reinterpret_cast<signed char*>(&q);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t mw = m[2 * k + (j >> 1)];
              if (tk + j >= r0 && tk + j < r1)
                e[j] = (signed char)quant(j & 1 ? bf_hi(mw) : bf_lo(mw), vrs);
              else if (tk + j < r0 && again)
                e[j] = (signed char)rintf(e[j] * vf);
            }
            *reinterpret_cast<char4*>(dst) = q;
          }
        }
      }
    }
    __syncthreads();  // the tiles are free for the next head
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
// bf16 in shared memory and read as transposed 8x8 tiles.
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
  if (i0 < nv) {
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
  const int64_t from = page_base(C, id, h) + at % C.P * D;
  const int64_t hs = (int64_t)id * C.H + h;
  bf16* tl = tile[warp];
  if constexpr (I8) {
    const float vs = C.vscale[hs];
#pragma unroll
    for (int dim = lane; dim < D; dim += 32) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<int8_t*>(C.v) + from + dim * kGroup);
      const signed char* e = reinterpret_cast<const signed char*>(&u);
      alignas(16) bf16 o[kGroup];
#pragma unroll
      for (int k = 0; k < kGroup; ++k) o[k] = __float2bfloat16_rn(e[k] * vs);
      *reinterpret_cast<uint4*>(tl + dim * kRow) = *reinterpret_cast<uint4*>(o);
      *reinterpret_cast<uint4*>(tl + dim * kRow + 8) = *reinterpret_cast<uint4*>(o + 8);
    }
  } else {
#pragma unroll
    for (int k = lane; k < 2 * D; k += 32)
      *reinterpret_cast<uint4*>(tl + (k >> 1) * kRow + (k & 1) * 8) =
          *reinterpret_cast<const uint4*>(static_cast<bf16*>(C.v) + from + k * 8);
  }
  const float ks = I8 ? C.kscale[hs] : 1.f;
#pragma unroll
  for (int k = lane; k < kGroup * (D / 8); k += 32) {
    const int r = k / (D / 8), piece = k % (D / 8);
    const int64_t i = i0 + r;
    if (i < 0 || i >= A.S.n) continue;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (i < nv) {
      if constexpr (I8) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<int8_t*>(C.k) + from + k * 8);
        const signed char* e = reinterpret_cast<const signed char*>(&w);
        alignas(16) bf16 o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __float2bfloat16_rn(e[j] * ks);
        u = *reinterpret_cast<uint4*>(o);
      } else {
        u = *reinterpret_cast<const uint4*>(static_cast<bf16*>(C.k) + from + k * 8);
      }
    }
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
