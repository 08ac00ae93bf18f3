// Host side of the rotary and cache entry points declared in
// include/lsh_attn.h: argument checks and launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "cache.cuh"
#include "cache_attend.cuh"
#include "lsh_attn.h"
#include "rope.cuh"
#include "tma_host.cuh"

namespace {

using namespace lsh;

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

inline lsh_status last_cuda() {
  return cudaGetLastError() == cudaSuccess ? LSH_OK : LSH_ERR_CUDA;
}

// Rows [B][H][n] of d contiguous elements: strides non-negative multiples of
// 16 bytes, and no axis steps further than 2^59 elements, so that sums of offsets in
// bytes stay below 2^63.
bool strides_ok(const int64_t (&s)[3], int B, int H, int n, int esize) {
  const int64_t count[3] = {B, H, n};
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] >= (int64_t(1) << 44) || s[i] * esize % 16 != 0 ||
        s[i] > (int64_t(1) << 59) / std::max<int64_t>(1, count[i] - 1))
      return false;
  return true;
}

// Whether rows that are written lie apart: sorted by stride, every axis steps
// over what the axes inside it span.
bool rows_apart(const int64_t (&s)[3], int B, int H, int n, int d) {
  std::pair<int64_t, int64_t> ax[3] = {{s[0], B}, {s[1], H}, {s[2], n}};
  std::sort(ax, ax + 3);
  int64_t span = d;  // elements from the first to one past the last so far
  for (const auto& a : ax) {
    if (a.second == 1) continue;
    if (a.first < span) return false;
    span += a.first * (a.second - 1);
  }
  return true;
}

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxBatch = 1 << 24;

// Checks `rot` and fills the plan. 0: no rotation is asked for.
lsh_status check_rot(const lsh_rope_axes* rot, int d, RotPlan* R) {
  *R = RotPlan{};
  if (!rot || rot->axes == 0) return LSH_OK;
  if (rot->axes < 0 || rot->axes > LSH_ROPE_MAX_AXES || (rot->adjacent != 0 && rot->adjacent != 1))
    return LSH_ERR_INVALID_ARG;
  int at = 0;
  for (int a = 0; a < rot->axes; ++a) {
    if (rot->dims[a] < 2 || rot->dims[a] % 2 != 0 || rot->dims[a] > d - at)
      return LSH_ERR_INVALID_ARG;
    R->off[a] = at;
    R->half[a] = rot->dims[a] / 2;
    at += rot->dims[a];
  }
  R->axes = rot->axes;
  R->adjacent = rot->adjacent;
  R->pairs = at / 2;
  return LSH_OK;
}

// Partners of halves lie in runs that have to stay inside their axis: the widest
// run, up to 16 bytes, that divides every axis's pairs (24 dimensions: 12 pairs,
// runs of 4).
int run_width(const RotPlan& R, int most) {
  int w = most;
  for (int a = 0; a < R.axes; ++a)
    while (R.half[a] % w != 0) w /= 2;
  return w;
}

template <typename T, int D>
lsh_status launch_rope(RopeArgs A, const void* x, void* out, cudaStream_t st) {
  constexpr int N = 16 / sizeof(T), kTok = 256 / (D / N);
  A.tiles = (A.n + kTok - 1) / kTok;
  // four blocks an SM or more are resident; heads are split over jobs where there
  // are fewer tiles
  const int64_t want = 4 * sm_count(), tiles = (int64_t)A.tiles * A.B;
  const int groups = (int)std::min<int64_t>(A.H, std::max<int64_t>(1, want / tiles));
  A.heads_per = (A.H + groups - 1) / groups;
  A.head_groups = (A.H + A.heads_per - 1) / A.heads_per;
  auto kern = k_rope<T, D, 1, false>;
  if (A.rot.adjacent) {
    kern = k_rope<T, D, 1, true>;
  } else {
    const int w = run_width(A.rot, N);
    if (w == N) kern = k_rope<T, D, N, false>;
    else if (w == 4) kern = k_rope<T, D, 4, false>;
    else if (w == 2) kern = k_rope<T, D, 2, false>;
  }
  // Neighbouring pairs: a job a block (0.89 of the copy rate at B1 H8 n65536 d128;
  // persistent blocks 0.84). Halves have more to work out before the first row:
  // persistent blocks (0.75 at B8 H8 n12288 d64, axes 24, 24, 16; a job a block 0.61).
  // (Measured with runs of four. Narrower ones have registers for two or three blocks an
  // SM only and take the same grid: 0.57 at axes 10, 14.)
  const int64_t jobs = tiles * A.head_groups;
  const int64_t most = A.rot.adjacent ? INT32_MAX : 5 * sm_count();
  const int64_t blocks = std::min(jobs, most), rest = blocks / A.tiles;
  A.step_tile = (int)(blocks % A.tiles);
  A.step_group = (int)(rest % A.head_groups);
  A.step_b = (int)(rest / A.head_groups);
  kern<<<(unsigned)blocks, 256, 0, st>>>(
      static_cast<const T*>(x), static_cast<T*>(out), A);
  return last_cuda();
}

// Shared memory of a kernel raised to `bytes`, once for each device: `done` is
// the kernel's own record. (The call costs about as much as a small launch.)
template <typename K>
bool allow_smem(K kern, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done->fetch_or(bit, std::memory_order_release);
  return true;
}

// ---------------------------------------------------------------- cache calls
lsh_status check_cache(const lsh_cache_desc* c, const lsh_cache* m, const lsh_cache_rows* r,
                       const int32_t* table, const int32_t* len, const int32_t* valid,
                       CacheView* C, SeqTables* S) {
  if (!c || !r) return LSH_ERR_INVALID_ARG;
  if (c->pages < 1 || c->heads < 1 || c->page_size < 1 || c->d < 1 ||
      (c->format != LSH_CACHE_BF16 && c->format != LSH_CACHE_I8) || r->batch < 1 || r->n < 1 ||
      r->max_pages < 1)
    return LSH_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || (c->page_size != 16 && c->page_size != 32 &&
                                      c->page_size != 64 && c->page_size != 128))
    return LSH_ERR_UNSUPPORTED;
  if (r->batch > 65535 || c->heads > 65535 || r->n > kMaxRows) return LSH_ERR_UNSUPPORTED;
  // positions are 32-bit, with the rows of a call behind them
  if ((int64_t)r->max_pages * c->page_size > INT32_MAX - kMaxRows) return LSH_ERR_UNSUPPORTED;
  if (!m) return LSH_OK;  // sizes only
  if (!m->k || !m->v || !m->key_inv_norm || !table || !len) return LSH_ERR_INVALID_ARG;
  if (c->format == LSH_CACHE_I8 && (!m->k_scale || !m->v_scale)) return LSH_ERR_INVALID_ARG;
  if (!aligned16(m->k) || !aligned16(m->v) || !aligned16(m->key_inv_norm) ||
      !aligned16(m->status))
    return LSH_ERR_INVALID_ARG;
  *C = CacheView{m->k,        m->v,          m->key_inv_norm,
                 m->k_scale,  m->v_scale,    static_cast<WsHeader*>(m->status),
                 c->pages,    c->heads,      c->page_size, c->d};
  *S = SeqTables{table, len, valid, r->batch, r->n, r->max_pages};
  return LSH_OK;
}

template <int D, bool I8, int R, int TURN>
lsh_status launch_append_t(const AppendArgs& A, cudaStream_t st) {
  constexpr int kBuf = append_buffers(D, R);
  auto kern = k_cache_append<D, I8, R, TURN>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, (int)append_smem(R, D, D / 2, kBuf), &done)) return LSH_ERR_CUDA;
  const int span = I8 && A.C.P > R ? A.C.P : R;  // tokens between blocks
  const dim3 grid((unsigned)((A.S.n + span - 2) / span + 1),
                  (unsigned)((A.C.H + A.heads_per - 1) / A.heads_per), (unsigned)A.S.B);
  kern<<<grid, append_threads(D, R), append_smem(R, D, A.rot.pairs, kBuf), st>>>(A);
  return last_cuda();
}

template <int D, bool I8, int R>
lsh_status launch_append_r(const AppendArgs& A, cudaStream_t st) {
  if (A.rot.axes == 0) return launch_append_t<D, I8, R, kTurnNone>(A, st);
  if (A.rot.adjacent) return launch_append_t<D, I8, R, kTurnAdjacent>(A, st);
  if (run_width(A.rot, 4) == 4) return launch_append_t<D, I8, R, kTurnRuns>(A, st);
  return launch_append_t<D, I8, R, kTurnSingles>(A, st);
}

template <int D>
lsh_status launch_append(const AppendArgs& A, bool i8, cudaStream_t st) {
  if (!i8) return launch_append_r<D, false, append_rows(false, 0, 0)>(A, st);
  switch (append_rows(true, A.C.P, A.S.n)) {
    case 32: return launch_append_r<D, true, 32>(A, st);
    case 64: return launch_append_r<D, true, 64>(A, st);
    default: return launch_append_r<D, true, 128>(A, st);
  }
}

// Workspace of the cached attention: for every segment a record, and for every
// computing warp two partial results of a segment's rows.
struct AttendLayout {
  int blocks, rows, groups;  // rows of a segment; segments of a (sequence, head)
  int64_t segments;
  size_t ml, part, total;
};

AttendLayout attend_layout(const lsh_cache_desc& c, const lsh_cache_rows& r) {
  AttendLayout L;
  L.blocks = sm_count();
  // calls of more than eight rows take sixteen together: the cache is read once for
  // them, and a product's other eight rows cost nothing
  L.rows = r.n > 8 ? 16 : 8;
  L.groups = (r.n + L.rows - 1) / L.rows;
  L.segments = (int64_t)r.batch * c.heads * L.groups;
  const int warps = c.d == 64 ? AttCfg<64, false>::kWarps : AttCfg<128, false>::kWarps;
  const size_t rows = (size_t)L.blocks * warps * 2 * L.rows;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  L.ml = up((size_t)L.segments * sizeof(int4));
  L.part = L.ml + up(rows * 2 * sizeof(float));
  L.total = L.part + up(rows * c.d * sizeof(float));
  return L;
}

template <int D, bool I8, int RG>
lsh_status launch_attend_rows(const AttendArgs& A, const AttendLayout& L, cudaStream_t st) {
  using Cfg = AttCfg<D, I8>;
  static_assert(Cfg::kWarps * Cfg::kDepth <= 32, "barriers");
  static_assert(sizeof(UnitMeta) <= 128 && Cfg::kStage % 16 == 0, "stage header");
  static_assert(Cfg::kSmem <= 227 * 1024, "shared memory");
  auto kern = k_cache_attend<D, I8, RG>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, Cfg::kSmem, &done)) return LSH_ERR_CUDA;
  kern<<<L.blocks, Cfg::kThreads, Cfg::kSmem, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return LSH_ERR_CUDA;
  // a table that holds one unit at most leaves nothing to join
  if ((int64_t)A.S.max_pages * A.C.P <= Cfg::kTok) return LSH_OK;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)L.segments, (unsigned)std::min(A.S.n, 8 * RG), D / 32);
  // a segment has about this many parts where it is shared at all
  const int64_t parts = (int64_t)L.blocks * Cfg::kWarps / L.segments + 2;
  cfg.blockDim = dim3(32u * (unsigned)std::min<int64_t>(8, (parts + 3) / 4));
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_cache_combine<D, 8 * RG>, A) == cudaSuccess ? LSH_OK : LSH_ERR_CUDA;
}

template <int D, bool I8>
lsh_status launch_attend(const AttendArgs& A, const AttendLayout& L, cudaStream_t st) {
  return L.rows == 8 ? launch_attend_rows<D, I8, 1>(A, L, st) : launch_attend_rows<D, I8, 2>(A, L, st);
}

}  // namespace

extern "C" {

lsh_status lsh_rope(const lsh_rope_desc* desc, const void* x, const int32_t* positions,
                    const float* freqs, void* out, void* stream) {
  if (!desc) return LSH_ERR_INVALID_ARG;
  const lsh_rope_desc& q = *desc;
  if (q.batch < 1 || q.heads < 1 || q.n < 1 || q.d < 1 || (q.inverse != 0 && q.inverse != 1) ||
      (q.pos_batched != 0 && q.pos_batched != 1) ||
      (q.dtype != LSH_F32 && q.dtype != LSH_BF16) || q.rot.axes < 1)
    return LSH_ERR_INVALID_ARG;
  if ((q.d != 64 && q.d != 128) || q.n > kMaxRows || q.batch > kMaxBatch || q.heads > 65535)
    return LSH_ERR_UNSUPPORTED;
  RopeArgs A;
  lsh_status s = check_rot(&q.rot, q.d, &A.rot);
  if (s != LSH_OK) return s;
  if (!x || !positions || !freqs || !out || !aligned16(x) || !aligned16(out))
    return LSH_ERR_INVALID_ARG;
  const int esize = q.dtype == LSH_BF16 ? 2 : 4;
  if (!strides_ok(q.x_stride, q.batch, q.heads, q.n, esize) ||
      !strides_ok(q.out_stride, q.batch, q.heads, q.n, esize) ||
      !rows_apart(q.out_stride, q.batch, q.heads, q.n, q.d))
    return LSH_ERR_INVALID_ARG;
  A.pos = positions;
  A.freqs = freqs;
  A.B = q.batch;
  A.H = q.heads;
  A.n = q.n;
  A.pos_axis = q.pos_batched ? (int64_t)q.batch * q.n : q.n;
  A.pos_batch = q.pos_batched ? q.n : 0;
  for (int i = 0; i < 3; ++i) {
    A.xs[i] = q.x_stride[i];
    A.os[i] = q.out_stride[i];
  }
  A.sign = q.inverse ? -1.f : 1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (q.dtype == LSH_BF16)
    return q.d == 64 ? launch_rope<__nv_bfloat16, 64>(A, x, out, st)
                     : launch_rope<__nv_bfloat16, 128>(A, x, out, st);
  return q.d == 64 ? launch_rope<float, 64>(A, x, out, st) : launch_rope<float, 128>(A, x, out, st);
}

lsh_status lsh_cache_append(const lsh_cache_desc* desc, const lsh_cache* cache,
                            const lsh_cache_rows* rows, const lsh_rope_axes* rot, const void* x,
                            const void* v, const int32_t* positions, const float* freqs,
                            const int32_t* page_table, const int32_t* seq_len,
                            const int32_t* n_valid, void* xr, void* stream) {
  if (!cache) return LSH_ERR_INVALID_ARG;
  AppendArgs A;
  lsh_status s = check_cache(desc, cache, rows, page_table, seq_len, n_valid, &A.C, &A.S);
  if (s != LSH_OK) return s;
  if ((s = check_rot(rot, A.C.d, &A.rot)) != LSH_OK) return s;
  if (!x || !v || !aligned16(x) || !aligned16(v) || !aligned16(xr)) return LSH_ERR_INVALID_ARG;
  if (A.rot.axes > 0 && (!positions || !freqs)) return LSH_ERR_INVALID_ARG;
  if (rows->pos_batched != 0 && rows->pos_batched != 1) return LSH_ERR_INVALID_ARG;
  if (!strides_ok(rows->x_stride, A.S.B, A.C.H, A.S.n, 2) ||
      !strides_ok(rows->v_stride, A.S.B, A.C.H, A.S.n, 2) ||
      (xr && (!strides_ok(rows->out_stride, A.S.B, A.C.H, A.S.n, 2) ||
              !rows_apart(rows->out_stride, A.S.B, A.C.H, A.S.n, A.C.d))))
    return LSH_ERR_INVALID_ARG;
  A.x = static_cast<const __nv_bfloat16*>(x);
  A.v = static_cast<const __nv_bfloat16*>(v);
  A.xr = static_cast<__nv_bfloat16*>(xr);
  A.pos = positions;
  A.freqs = freqs;
  A.pos_axis = rows->pos_batched ? (int64_t)A.S.B * A.S.n : A.S.n;
  A.pos_batch = rows->pos_batched ? A.S.n : 0;
  for (int i = 0; i < 3; ++i) {
    A.xs[i] = rows->x_stride[i];
    A.vs[i] = rows->v_stride[i];
    A.os[i] = rows->out_stride[i];
  }
  const bool i8 = desc->format == LSH_CACHE_I8;
  const int rows_per = append_rows(i8, A.C.P, A.S.n), span = i8 ? std::max(A.C.P, rows_per) : rows_per;
  const int64_t blocks = (int64_t)((A.S.n + span - 2) / span + 1) * A.S.B;
  // heads are split over blocks until these fill the card twice: every block forms
  // its tokens' angles again (8 int8 sequences of up to 2000 rows, H8 d64: 25 us; once
  // 35, three times 28)
  const int threads = append_threads(A.C.d, rows_per);
  const int64_t want = 2 * (1024 / threads) * sm_count();
  const int groups = (int)std::min<int64_t>(A.C.H, std::max<int64_t>(1, want / blocks));
  A.heads_per = (A.C.H + groups - 1) / groups;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return A.C.d == 64 ? launch_append<64>(A, i8, st) : launch_append<128>(A, i8, st);
}

lsh_status lsh_cache_gather(const lsh_cache_desc* desc, const lsh_cache* cache,
                            const lsh_cache_rows* rows, const int32_t* page_table,
                            const int32_t* start, const int32_t* n_valid, void* x, void* v,
                            void* stream) {
  if (!cache) return LSH_ERR_INVALID_ARG;
  GatherArgs A;
  lsh_status s = check_cache(desc, cache, rows, page_table, start, n_valid, &A.C, &A.S);
  if (s != LSH_OK) return s;
  if (!x || !v || !aligned16(x) || !aligned16(v)) return LSH_ERR_INVALID_ARG;
  if (!strides_ok(rows->x_stride, A.S.B, A.C.H, A.S.n, 2) ||
      !strides_ok(rows->v_stride, A.S.B, A.C.H, A.S.n, 2) ||
      !rows_apart(rows->x_stride, A.S.B, A.C.H, A.S.n, A.C.d) ||
      !rows_apart(rows->v_stride, A.S.B, A.C.H, A.S.n, A.C.d))
    return LSH_ERR_INVALID_ARG;
  A.x = static_cast<__nv_bfloat16*>(x);
  A.v = static_cast<__nv_bfloat16*>(v);
  for (int i = 0; i < 3; ++i) {
    A.xs[i] = rows->x_stride[i];
    A.vs[i] = rows->v_stride[i];
  }
  A.groups = (A.S.n + kGroup - 2) / kGroup + 1;
  const dim3 grid((unsigned)((A.groups + 7) / 8), (unsigned)A.C.H, (unsigned)A.S.B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = desc->format == LSH_CACHE_I8;
  auto kern = A.C.d == 64 ? (i8 ? k_cache_gather<64, true> : k_cache_gather<64, false>)
                          : (i8 ? k_cache_gather<128, true> : k_cache_gather<128, false>);
  kern<<<grid, 256, 0, st>>>(A);
  return last_cuda();
}

lsh_status lsh_cache_attend_workspace_size(const lsh_cache_desc* desc, const lsh_cache_rows* rows,
                                           size_t* bytes) {
  lsh_status s = check_cache(desc, nullptr, rows, nullptr, nullptr, nullptr, nullptr, nullptr);
  if (s != LSH_OK) return s;
  if (!bytes) return LSH_ERR_INVALID_ARG;
  const AttendLayout L = attend_layout(*desc, *rows);
  if (L.segments > INT32_MAX) return LSH_ERR_UNSUPPORTED;
  *bytes = L.total;
  return LSH_OK;
}

lsh_status lsh_cache_attend(const lsh_cache_desc* desc, const lsh_cache* cache,
                            const lsh_cache_rows* rows, const void* x, const int32_t* page_table,
                            const int32_t* seq_len, const int32_t* n_valid, void* out, float* lse,
                            void* ws, size_t ws_bytes, void* stream) {
  if (!cache) return LSH_ERR_INVALID_ARG;
  AttendArgs A;
  lsh_status s = check_cache(desc, cache, rows, page_table, seq_len, n_valid, &A.C, &A.S);
  if (s != LSH_OK) return s;
  if (!x || !out || !lse || !aligned16(x) || !aligned16(out)) return LSH_ERR_INVALID_ARG;
  if (!strides_ok(rows->x_stride, A.S.B, A.C.H, A.S.n, 2) ||
      !strides_ok(rows->out_stride, A.S.B, A.C.H, A.S.n, 2) ||
      !rows_apart(rows->out_stride, A.S.B, A.C.H, A.S.n, A.C.d))
    return LSH_ERR_INVALID_ARG;
  const AttendLayout L = attend_layout(*desc, *rows);
  if (L.segments > INT32_MAX) return LSH_ERR_UNSUPPORTED;
  if (!ws || ((uintptr_t)ws & 255) != 0 || ws_bytes < L.total) return LSH_ERR_WORKSPACE;
  A.x = static_cast<const __nv_bfloat16*>(x);
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  for (int i = 0; i < 3; ++i) {
    A.xs[i] = rows->x_stride[i];
    A.os[i] = rows->out_stride[i];
  }
  unsigned char* w = static_cast<unsigned char*>(ws);
  A.groups = L.groups;
  A.rec = reinterpret_cast<int4*>(w);
  A.part_ml = reinterpret_cast<float*>(w + L.ml);
  A.part = reinterpret_cast<float*>(w + L.part);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = desc->format == LSH_CACHE_I8;
  if (A.C.d == 64) return i8 ? launch_attend<64, true>(A, L, st) : launch_attend<64, false>(A, L, st);
  return i8 ? launch_attend<128, true>(A, L, st) : launch_attend<128, false>(A, L, st);
}

}  // extern "C"
