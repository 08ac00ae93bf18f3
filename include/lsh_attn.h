/*
 * lsh_attn.h -- C ABI of the B200 (sm_100a) Reformer shared-QK LSH-attention
 * forward pass.
 *
 * The method (sources are web pages on Reformer, cited by title and section):
 *   - hash: for b buckets a random R of size [dimension, b/2] maps x to
 *     argmax([xR ; -xR])                  ("Reformer summary", §局部敏感哈希)
 *   - several independent hash rounds     ("Reformer summary", §多輪LSH哈希)
 *   - sort the tokens by bucket, then by position; cut the sorted order into
 *     chunks of m and attend inside them  ("Reformer summary", §局部敏感哈希注意力)
 *   - keys are the shared vectors scaled to unit length, logits are scaled by
 *     1/sqrt(d) ("Reformer: LSH attention and reversible layers", §二.1)
 *   - a token attends to itself only when nothing else is available
 *                                         ("Reformer summary", §共享QK中的自掩碼)
 * Readings taken where the pages are silent: a query in chunk c sees the keys
 * of chunks c-1 and c (chunk 0 sees only itself); the self logit is -1e5;
 * causal masking removes keys at later positions; rounds are merged by
 * weighting each round's output with exp(lse_r - logsumexp_r lse_r); argmax
 * ties go to the first index of [xR ; -xR].
 *
 * Conventions for every entry point
 *   - All array pointers are DEVICE pointers owned by the caller. The library
 *     never allocates device memory; scratch space is the caller's workspace of
 *     at least lsh_attn_workspace_size() bytes, 256-byte aligned.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *     default stream) and never synchronise the host, except
 *     lsh_attn_get_device_status / lsh_attn_get_diag, which synchronise
 *     `stream`.
 *   - Argument errors are detected on the host before anything is launched;
 *     nothing is written then. Errors found by the kernels (a caller bucket id
 *     outside [0, n_buckets), a bounded wait that gave up) are recorded in the
 *     workspace status word and read with lsh_attn_get_device_status.
 *   - Results are deterministic: identical inputs give bit-identical outputs.
 *   - One workspace must not be shared by calls that may run concurrently.
 *
 * Layouts (row-major, innermost last; B batch, H heads, n length, d head
 * dim, nb buckets, Rn rounds):
 *   x, v, out    [B][H][n][d]          in desc.dtype
 *   R            [Rn][d][nb/2]         in desc.dtype
 *   buckets      [B][H][Rn][n]         int32, position order
 *   perm         [B][H][Rn][n]         int32: perm[s] = position at sorted slot s
 *   xs, vs       [B][H][Rn][n][d]      desc.dtype, rows in sorted order
 *   lse          [B][H][Rn][n]         fp32, position order, natural log
 *
 * Supported (else LSH_ERR_UNSUPPORTED): dtype LSH_F32 or LSH_BF16; d in
 * {64, 128}; n_buckets even with 2 <= n_buckets <= 4096; chunk m >= 1 with
 * min(m, n) <= 128 and n % min(m, n) == 0 (m >= n is a single chunk);
 * 1 <= rounds <= 16; n * n_buckets < 2^31.
 */
#ifndef LSH_ATTN_H
#define LSH_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LSH_OK = 0,
    LSH_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad enum */
    LSH_ERR_UNSUPPORTED = 2, /* a valid problem outside the supported set */
    LSH_ERR_WORKSPACE = 3,   /* workspace missing, misaligned or too small */
    LSH_ERR_CUDA = 4,        /* a CUDA runtime call failed */
    LSH_ERR_TIMEOUT = 5,     /* a kernel's bounded wait gave up */
    LSH_ERR_DEVICE = 6       /* a kernel rejected its input (bucket id range) */
} lsh_status;

typedef enum { LSH_F32 = 0, LSH_BF16 = 1 } lsh_dtype;

/* Problem description shared by every call. */
typedef struct {
    int32_t batch;     /* B >= 1 */
    int32_t heads;     /* H >= 1 */
    int32_t n;         /* sequence length >= 1 */
    int32_t d;         /* head dimension */
    int32_t n_buckets; /* nb: even, buckets per round */
    int32_t chunk;     /* m: chunk length in the sorted order */
    int32_t rounds;    /* independent hash rounds */
    int32_t causal;    /* 0 or 1 */
    int32_t dtype;     /* lsh_dtype of x, v, R, out, xs, vs */
} lsh_attn_desc;

/* Counters written by the kernels into the workspace header; reset at the
 * start of every hash / sort / forward call. */
typedef struct {
    uint32_t status;         /* lsh_status recorded by a kernel, 0 if none */
    uint32_t hash_refined;   /* (token, round) hashes re-decided in fp64 */
    uint32_t bad_bucket_ids; /* caller bucket ids outside [0, nb), clamped */
    uint32_t reserved;
} lsh_attn_diag;

/* Workspace bytes that lsh_attn_hash / lsh_attn_sort / lsh_attn_forward need
 * for `desc`. Writes *bytes; errors as for the calls themselves. */
lsh_status lsh_attn_workspace_size(const lsh_attn_desc *desc, size_t *bytes);

/* Hash every token in every round ("Reformer summary", §局部敏感哈希 and
 * §多輪LSH哈希): buckets[b][h][r][i] = argmax([x_i R_r ; -x_i R_r]), first
 * index on ties, bit-exact to the fp64 definition (bf16 runs on tensor cores
 * and re-decides near ties in fp64; fp32 runs in fp64).
 * x [B][H][n][d], R [Rn][d][nb/2] in desc.dtype; buckets out, int32. */
lsh_status lsh_attn_hash(const lsh_attn_desc *desc, const void *x, const void *R,
                         int32_t *buckets, void *workspace, size_t workspace_bytes,
                         void *stream);

/* Stable sort of every (batch, head, round) by bucket, then position
 * ("Reformer summary", §局部敏感哈希注意力): perm[s] = the position at sorted
 * slot s. If x, v, xs and vs are all non-NULL the rows of x and v are also
 * gathered into sorted order: xs[..][s] = x[..][perm[s]]; pass all four NULL
 * to skip the gather. buckets [B][H][Rn][n] int32 in [0, nb) (ids outside are
 * clamped and counted in the diag). */
lsh_status lsh_attn_sort(const lsh_attn_desc *desc, const int32_t *buckets, const void *x,
                         const void *v, int32_t *perm, void *xs, void *vs, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Whole forward pass: hash (skipped when `buckets` is non-NULL: the caller's
 * ids are used as given), sort and gather, chunked attention with unit keys,
 * 1/sqrt(d) scale, optional causal mask and the -1e5 self logit, un-sort, and
 * the logsumexp round merge. out [B][H][n][d] in desc.dtype; lse [B][H][Rn][n]
 * fp32 holds every round's log-normaliser in position order. */
lsh_status lsh_attn_forward(const lsh_attn_desc *desc, const void *x, const void *v,
                            const void *R, const int32_t *buckets, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Number of events lsh_attn_forward_profiled records. */
#define LSH_ATTN_PROFILE_EVENTS 10

/* lsh_attn_forward that also records the caller's CUDA events on `stream`
 * at every kernel boundary, for timing each kernel on the device:
 *   [0] start               [1] after the rotation transpose of the hash
 *   [2] after the projection / argmax kernel  [3] after the fp64 re-decision
 *   [4] after the bucket histograms  [5] after their scan
 *   [6] after the stable ranks (perm/inv)  [7] after the row gather
 *   [8] after the chunked attention  [9] after the un-sort and round merge
 * A kernel that does not run for this problem (caller-supplied buckets, the
 * fp64 hash) leaves consecutive events with nothing between them.
 * `events` points to LSH_ATTN_PROFILE_EVENTS cudaEvent_t handles created by
 * the caller. */
lsh_status lsh_attn_forward_profiled(const lsh_attn_desc *desc, const void *x, const void *v,
                                     const void *R, const int32_t *buckets, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, void *stream,
                                     void *const *events);

/* Synchronise `stream` and return the status the kernels recorded in
 * `workspace` since the last call that used it (LSH_OK if none). */
lsh_status lsh_attn_get_device_status(const void *workspace, void *stream);

/* Synchronise `stream` and copy the workspace counters into *diag. */
lsh_status lsh_attn_get_diag(const void *workspace, void *stream, lsh_attn_diag *diag);

/* Self-test of the bounded waits every kernel uses: clears the workspace
 * status word, then launches one CTA that waits on an mbarrier nothing
 * arrives at, with a limit of `limit_us` microseconds (1 .. 2000000) instead
 * of the kernels' 2 s. The wait gives up, the kernel records LSH_ERR_TIMEOUT
 * in the status word and returns, and the stream stays usable: read the
 * status with lsh_attn_get_device_status. `workspace` needs at least 256
 * bytes. Returns LSH_ERR_INVALID_ARG for a null workspace, too small a size
 * or a limit out of range (nothing is launched then). */
lsh_status lsh_attn_selftest_wait_timeout(void *workspace, size_t workspace_bytes,
                                          uint32_t limit_us, void *stream);

/* Size of the device-resident scratch of lsh_attn_sort_noalloc (8 MiB). */
#define LSH_ATTN_NOALLOC_SCRATCH_BYTES (8u << 20)

/* The stable sort of lsh_attn_sort (perm only, no row gather) for callers
 * that must not allocate device memory and cannot pass a workspace: for
 * example a plug-in whose host runtime owns all device memory, or a loop that
 * cannot afford the device synchronisation of cudaMalloc / cudaFree. The
 * paper has no counterpart to this entry point; it only changes where the
 * scratch lives. No memory is allocated: the scratch is a fixed array of
 * LSH_ATTN_NOALLOC_SCRATCH_BYTES in the library's own device memory, held by
 * every GPU that loads the library until the process exits.
 *   - buckets [B][H][Rn][n] int32 in; perm [B][H][Rn][n] int32 out (device).
 *   - A problem needs 256 + 4*B*H*Rn*nb*ceil(n / T) (rounded up to 256) +
 *     4*B*H*Rn*n bytes of scratch, T = 256 * clamp(8192 / nb, 1, 8); larger
 *     problems return LSH_ERR_UNSUPPORTED and write nothing (use lsh_attn_sort).
 *   - The first call on a device looks up the scratch's device address (with
 *     that device current) and caches it for the life of the process; make
 *     that first call before any stream capture. cudaDeviceReset on a device
 *     makes the cached address stale: after a reset, do not call this entry
 *     point on that device again in the same process.
 *   - Every call on a device shares the one scratch, whose contents persist
 *     from the previous call: calls that may overlap on the GPU (different
 *     streams without ordering between them) race and must not be issued.
 *   - Host-side errors as for lsh_attn_sort. The kernels' status word lives
 *     in the shared scratch and no call reads it, so bucket ids outside
 *     [0, nb) are clamped into range SILENTLY here (the perm is that of the
 *     clamped ids and the call returns LSH_OK); lsh_attn_sort reports the
 *     same input as LSH_ERR_DEVICE. */
lsh_status lsh_attn_sort_noalloc(const lsh_attn_desc *desc, const int32_t *buckets,
                                 int32_t *perm, void *stream);

/* Workspace bytes lsh_attn_dense_forward needs for `desc` (only batch,
 * heads, n, d, causal and dtype are read). Writes *bytes. */
lsh_status lsh_attn_dense_workspace_size(const lsh_attn_desc *desc, size_t *bytes);

/* Dense shared-QK attention, the full-attention baseline the pages compare
 * LSH attention with ("Reformer: LSH attention and reversible layers",
 * §三.3): every query attends to every key (causal: every key at an earlier
 * position) under the same rules as lsh_attn_forward's chunks -- keys scaled
 * to unit length, logits scaled by 1/sqrt(d), the -1e5 self logit -- so it
 * equals lsh_attn_forward with one round and one chunk spanning the sequence.
 *   x, v, out [B][H][n][d] bf16 (LSH_BF16 only, else LSH_ERR_UNSUPPORTED);
 *   lse [B][H][n] fp32, natural log. Any n >= 1; d in {64, 128};
 *   B * H * roundup(n, 128) < 2^31. n_buckets, chunk and rounds are ignored.
 *   workspace: lsh_attn_dense_workspace_size bytes, 256-byte aligned.
 * Conventions (ownership, asynchrony, errors) as for lsh_attn_forward. */
lsh_status lsh_attn_dense_forward(const lsh_attn_desc *desc, const void *x, const void *v,
                                  void *out, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Workspace bytes lsh_attn_backward needs for `desc`. Writes *bytes. */
lsh_status lsh_attn_backward_workspace_size(const lsh_attn_desc *desc, size_t *bytes);

/* Gradients of lsh_attn_forward with respect to x and v, for training
 * ("Reformer re-reading", §2.2, trains the model end to end). Bucket ids are
 * an input, as in the forward they were computed from (the hash is piecewise
 * constant and is not differentiated), and the sort is recomputed from them.
 *   x, v [B][H][n][d]; buckets [B][H][Rn][n]; out [B][H][n][d] and lse
 *   [B][H][Rn][n] from the forward on those inputs; dout = dL/dout
 *   [B][H][n][d]; dlse = dL/dlse [B][H][Rn][n] fp32 or NULL (zero);
 *   dx, dv [B][H][n][d] out. x, v, out, dout, dx, dv in desc.dtype.
 * Supported: LSH_BF16 with chunk 64 and n % 64 == 0 (else
 * LSH_ERR_UNSUPPORTED); other limits as for lsh_attn_forward.
 * The gradient is that of the definition: the self logit and masked keys
 * carry none, and the rounds' merge weights are differentiated; the round
 * outputs themselves are not needed (their term cancels). Deterministic.
 * Conventions (ownership, asynchrony, errors) as for lsh_attn_forward;
 * bucket ids outside [0, nb) are clamped and reported as there. */
lsh_status lsh_attn_backward(const lsh_attn_desc *desc, const void *x, const void *v,
                             const int32_t *buckets, const void *out, const float *lse,
                             const void *dout, const float *dlse, void *dx, void *dv,
                             void *workspace, size_t workspace_bytes, void *stream);

/* A reversible layer around the attention ("Reformer: LSH attention and
 * reversible layers", §二.2 reversible residual and §二.3 chunked
 * feed-forward): with x = [x1, x2],
 *   y1 = x1 + Attn(x2),   y2 = x2 + FFN(y1),
 * and back:  x2 = y2 - FFN(y1),   x1 = y1 - Attn(x2).
 * Attn(x) = W_o applied to the heads of lsh_attn_forward(x W_qk^T, x W_v^T)
 * (shared QK, d_model = heads * d_head), FFN(y) = max(y W1^T + b1, 0) W2^T
 * + b2 computed ffn_chunk rows at a time (the rows are independent, so the
 * chunk only bounds the intermediate buffer). */
typedef struct {
    int32_t batch, n;        /* sequences and their length (n % 128 == 0) */
    int32_t d_model;         /* = heads * d_head, a multiple of 128 */
    int32_t heads, d_head;   /* d_head in {64, 128} */
    int32_t d_ff;            /* feed-forward width, a multiple of 128 */
    int32_t ffn_chunk;       /* rows per feed-forward chunk, a multiple of 128 */
    int32_t n_buckets, chunk, rounds, causal;  /* the attention's (chunk 64) */
    int32_t hash_buckets;    /* forward: 1 = hash into `buckets`, 0 = read them */
} lsh_rev_desc;

/* Weights, bf16 stored out x in (row j holds output feature j), biases fp32
 * (either may be NULL for zero). */
typedef struct {
    const void *w_qk, *w_v, *w_o;  /* [d_model][d_model] */
    const void *w1;                /* [d_ff][d_model] */
    const float *b1;               /* [d_ff] */
    const void *w2;                /* [d_model][d_ff] */
    const float *b2;               /* [d_model] */
} lsh_rev_weights;

/* Workspace bytes lsh_rev_block needs for `desc`. */
lsh_status lsh_rev_workspace_size(const lsh_rev_desc *desc, size_t *bytes);

/* inverse = 0: (in1, in2) = (x1, x2) -> (out1, out2) = (y1, y2); the bucket
 * ids [batch][heads][rounds][n] are hashed from x2 W_qk^T under R into
 * `buckets` (desc.hash_buckets = 1) or read from it (0).
 * inverse = 1: (in1, in2) = (y1, y2) -> (out1, out2) = (x1, x2) with the
 * forward's bucket ids read from `buckets` (R unused).
 * All activations [batch][n][d_model] bf16, device memory, 16-byte aligned.
 * Kernel status (the products' and the attention's) is read with
 * lsh_attn_get_device_status(workspace). Other conventions as for
 * lsh_attn_forward. */
lsh_status lsh_rev_block(const lsh_rev_desc *desc, int inverse, const void *in1, const void *in2,
                         const lsh_rev_weights *weights, const void *R, int32_t *buckets,
                         void *out1, void *out2, void *workspace, size_t workspace_bytes,
                         void *stream);

/* The in-bucket top-k variant of LSH attention ("Reformer re-reading",
 * §2.2), a second workload beside lsh_attn_forward: per round l, bucket(x) =
 * (sum_t [proj_l[:, t] . x > 0] 2^t) mod n_buckets over n_bits projections;
 * every query ranks the keys of its bucket (causal: positions <= its own) by
 * the chunked attention's logit x_i . x_j / (||x_j|| sqrt(d)) (-1e5 for
 * itself; higher first, lower position on ties) and keeps the top_k; the
 * candidates are the union over rounds, attended with one softmax of those
 * logits. Bucket bits and top-k sets are decided in fp64 (sums in increasing
 * feature order, no fused multiply-add); the softmax runs in fp32. */
typedef struct {
    int32_t batch, heads, n, d;  /* d in {64, 128} */
    int32_t n_buckets;           /* K: even, 2 .. 4096 */
    int32_t n_bits;              /* m projections per round, 1 .. 32 */
    int32_t top_k;               /* 1 .. 32 */
    int32_t rounds;              /* L: 1 .. 8 */
    int32_t causal;
} lsh_topk_desc;

/* Workspace bytes lsh_topk_forward needs for `desc`. */
lsh_status lsh_topk_workspace_size(const lsh_topk_desc *desc, size_t *bytes);

/* x, v, out [B][H][n][d] bf16; proj [rounds][d][n_bits] bf16; lse [B][H][n]
 * fp32; cand (optional, else kept in the workspace) [B][H][rounds][n][top_k]
 * int32: each round's top-k positions, best first, -1 past the kept ones.
 * Conventions as for lsh_attn_forward. */
lsh_status lsh_topk_forward(const lsh_topk_desc *desc, const void *x, const void *v,
                            const void *proj, void *out, float *lse, int32_t *cand,
                            void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions with one to four axes, a paged cache of shared-QK rows and
 * values, and attention of new tokens over it: what generating from a causal
 * shared-QK model needs beside the forward pass. Positions inside the shared
 * vectors and a cache have no counterpart on the pages; the attention keeps
 * their rules (unit keys, 1/sqrt(d), a token sees itself only when alone).
 *
 * Conventions as above, and for the calls below
 *   - Rows are given with three strides, in elements, for (batch, head,
 *     position); the d values of a row are contiguous. Row pointers are
 *     16-byte aligned and strides multiples of 16 bytes, so both
 *     [B][H][n][d] and the projections' [B][n][H][d] are read in place.
 *     Strides of inputs may be 0 (one row for all), no axis may step further than
 *     2^59 elements, and written rows must not overlap (LSH_ERR_INVALID_ARG).
 *     Limits (else LSH_ERR_UNSUPPORTED): n, the rows of a sequence, and the
 *     batch of lsh_rope 2^24; heads and the batches of the cache's calls 65535;
 *     max_pages * page_size 2^31 - 2^24.
 *   - Lengths, page numbers and positions are read on the device: a captured
 *     graph may be replayed after they change.
 *   - Nothing is allocated and no call synchronises.
 */
#define LSH_ROPE_MAX_AXES 4

/* How a row's dimensions are rotated. Axis a turns the dims[a] dimensions
 * after those of the axes before it, in dims[a] / 2 pairs; dimensions after
 * the last axis are left as they are. */
typedef struct {
    int32_t axes;                    /* 1 .. 4 (lsh_cache_append: 0 = no rotation) */
    int32_t dims[LSH_ROPE_MAX_AXES]; /* even, >= 2, sum <= d */
    int32_t adjacent; /* pair i of an axis: its dimensions 2i and 2i + 1 (1),
                       * or i and i + dims / 2 (0) */
} lsh_rope_axes;

typedef struct {
    int32_t batch, heads, n, d;  /* d in {64, 128} */
    int32_t dtype;               /* lsh_dtype of x and out */
    int32_t inverse;             /* 1: rotate by the negative angles */
    int32_t pos_batched;         /* positions [axes][batch][n] (1) or [axes][n] (0) */
    lsh_rope_axes rot;
    int64_t x_stride[3], out_stride[3];
} lsh_rope_desc;

/* Rotary positions: pair (lo, hi) of axis a, the p-th pair of all, turns by
 * t = positions[a] * freqs[p]:
 *   out[lo] = x[lo] cos t - x[hi] sin t,  out[hi] = x[lo] sin t + x[hi] cos t.
 * The angle is formed as a fraction of a turn in 64 bits, so far positions keep
 * their precision; the rotation is fp32 and rounds once. inverse = 1 is the
 * gradient with respect to x (and undoes the call). Sines and cosines of bf16
 * rows are good to 2^-21, of fp32 rows to 2^-23. positions int32, any sign;
 * freqs [sum dims / 2] fp32, any sign, at most 2^45 in size. out may be x
 * itself with the same strides, else they must not overlap. */
lsh_status lsh_rope(const lsh_rope_desc *desc, const void *x, const int32_t *positions,
                    const float *freqs, void *out, void *stream);

typedef enum { LSH_CACHE_BF16 = 0, LSH_CACHE_I8 = 1 } lsh_cache_format;

/* A paged cache. A page holds page_size consecutive tokens of one sequence
 * for every head. */
typedef struct {
    int32_t pages;      /* pages in the pool */
    int32_t heads;
    int32_t page_size;  /* 16, 32, 64 or 128 tokens */
    int32_t d;          /* 64 or 128 */
    int32_t format;     /* lsh_cache_format */
} lsh_cache_desc;

/* Its memory, 16-byte aligned, owned by the caller:
 *   k   [pages][heads][page_size][d]           rows of x, bf16 or int8
 *   v   [pages][heads][page_size / 16][d][16]  values, bf16 or int8: groups of
 *       16 tokens, dimension-major inside (the order the attention's P V
 *       product reads)
 *   key_inv_norm [pages][heads][page_size]     fp32, 1/||x|| (0 below 2^-126)
 *   k_scale, v_scale [pages][heads]            fp32, int8 only: a power of two
 *       s for each page and head; a stored q stands for q * s
 *   status  NULL, or at least 256 bytes, zeroed by the caller: the kernels
 *       record the first error they meet (LSH_ERR_DEVICE) and leave it until
 *       the caller clears it; lsh_attn_get_device_status reads it. */
typedef struct {
    void *k, *v;
    float *key_inv_norm, *k_scale, *v_scale;
    void *status;
} lsh_cache;

/* Rows that a call appends, reads back or attends from. */
typedef struct {
    int32_t batch;      /* sequences, at most 65535 */
    int32_t n;          /* rows of each (padded batch: the most) */
    int32_t max_pages;  /* columns of page_table */
    int32_t pos_batched;              /* lsh_cache_append: as in lsh_rope_desc */
    int64_t x_stride[3], v_stride[3]; /* x / out and v (lsh_cache_attend: x only) */
    int64_t out_stride[3];            /* xr, or the attention's out */
} lsh_cache_rows;

/* Tables of the calls below, int32 on the device: page_table
 * [batch][max_pages], the page of each page_size tokens of a sequence (only
 * the entries of tokens that are read or written count); seq_len [batch], the
 * tokens that a sequence holds before the call's n rows; n_valid [batch], how
 * many of the n rows each sequence has (NULL: all n). A sequence with
 * seq_len < 0, n_valid outside [0, n] or more tokens than max_pages pages
 * hold is taken to have no rows, and a page number outside [0, pages) to hold
 * nothing: neither is read or written, and both are recorded in the status. */

/* Append rows seq_len .. seq_len + n_valid - 1 of every sequence: x, rotated
 * by `rot` (as lsh_rope, result rounded to bf16; rot->axes 0 or rot NULL: as
 * it is), and v, both bf16; 1/||x|| is taken of the row as it is given. xr,
 * unless NULL, receives the rotated rows (the queries of lsh_cache_attend),
 * zeros past n_valid. Slots of other tokens are left as they are.
 * int8: a page's scale is the smallest power of two s >= 2^-126 such that
 * 127 s covers the finite values of the rows it was given since its first; rows
 * that raise it have the earlier rows of the page rounded again from what is
 * stored, q' = rint(q s / s'). The first row of a page sets its scale afresh;
 * while a page holds earlier rows, its scale never falls. So rows that are
 * overwritten later (drafted ones, by a call with a smaller seq_len) count in the
 * scale and in the rounding of those before them for good. Infinities are stored as
 * +-127 s, NaN as 0, and recorded in the status; a row of x that has one gets
 * key_inv_norm 0, so that its logits are 0 and it spoils no other token.
 * A page that is written must belong to one sequence of the call and stand in
 * its table once; a prefix that several sequences share may be read by all. */
lsh_status lsh_cache_append(const lsh_cache_desc *desc, const lsh_cache *cache,
                            const lsh_cache_rows *rows, const lsh_rope_axes *rot, const void *x,
                            const void *v, const int32_t *positions, const float *freqs,
                            const int32_t *page_table, const int32_t *seq_len,
                            const int32_t *n_valid, void *xr, void *stream);

/* Read rows start .. start + n_valid - 1 of every sequence back as values:
 * x (rotated as they were stored) and v, bf16 with x_stride and v_stride;
 * rows past n_valid, and those of bad pages, are zeros. `start` takes the
 * place of seq_len. For lsh_attn_forward over cached tokens, among others. */
lsh_status lsh_cache_gather(const lsh_cache_desc *desc, const lsh_cache *cache,
                            const lsh_cache_rows *rows, const int32_t *page_table,
                            const int32_t *start, const int32_t *n_valid, void *x, void *v,
                            void *stream);

/* Workspace bytes of lsh_cache_attend (256-byte aligned; contents need not be
 * kept or cleared between calls). */
lsh_status lsh_cache_attend_workspace_size(const lsh_cache_desc *desc,
                                           const lsh_cache_rows *rows, size_t *bytes);

/* Attention of the n newest tokens of every sequence, whose rows
 * lsh_cache_append has stored: token t (0 .. n_valid - 1) at position
 * p = seq_len + t sees every cached token j <= p with the logit
 *   x_t . k_j key_inv_norm_j / sqrt(d),   and -1e5 for itself (j = p),
 * as lsh_attn_dense_forward does with causal = 1; x are the (rotated) rows in
 * bf16, k_j and v_j the cache's values. Products x_t . k_j are fp32 sums of the
 * rows as they are: ||x_t|| ||x_j|| has to stay below 2^100. Weights times values are
 * fp32 sums too, of weights to 2^-17 of each (of an int8 page whose v_scale lies 2^100
 * below another's, values may count as zeros).
 *   out bf16 (out_stride), lse [batch][heads][n] fp32, natural log.
 * Rows past n_valid, and rows that see nothing (bad pages), are zeros with
 * lse = -inf. Made for few tokens a sequence (one, or a handful of drafted
 * ones): up to sixteen rows read the cache once. Deterministic on one device. */
lsh_status lsh_cache_attend(const lsh_cache_desc *desc, const lsh_cache *cache,
                            const lsh_cache_rows *rows, const void *x,
                            const int32_t *page_table, const int32_t *seq_len,
                            const int32_t *n_valid, void *out, float *lse, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Static, human-readable name of a status code. */
const char *lsh_attn_status_string(lsh_status status);

#ifdef __cplusplus
}
#endif

#endif /* LSH_ATTN_H */
