/*
 * tgemm — fused tensor-core GEMM with an in-kernel epilogue, for GB300 (sm_103a).
 *
 *     C[i, j] = epi( sum_{k<K} A[i, k] * B[k, j]  (+ bias[j]) )    0 <= i < M, 0 <= j < N
 *
 * The operation is the GEMM of "从零开始学习 TileLang：从 Python、PyTorch 到高性能
 * GPU Kernel 的完整开发教程", ch.10 §10.1 (C_ij = sum_k A_ik B_kj, 2MNK flops,
 * §10.9), with the epilogue of its §10.8 "GEMM Epilogue 融合" (relu(a @ b + bias),
 * bias indexed by the output column, applied before the write-back), the
 * C = ReLU(A @ B) kernel of "Writing high-performance kernels in TileLang"
 * ("Écrivons un GEMM"), the Bias (N,) operand of "TileLang で GPU カーネル設計を
 * 解説" §4, and the load -> GEMM -> activation -> store tile fusion of
 * "【CUDA】TileFusion".  Precision follows the tutorial's §10.7 recipe: fp16 or
 * bf16 inputs, tensor-core products, fp32 accumulation, one final rounding to
 * the input dtype (round to nearest even).  ReLU maps x <= 0 (including -0.0)
 * to +0.0 and keeps NaN.  The GELU epilogue (below) is the bias + GELU fusion
 * of "TileLang で GPU カーネル設計を解説" §4.
 *
 * Layout: every matrix is row-major with an explicit leading dimension (row
 * pitch, in elements): A[i, k] at A + i*lda + k, B[k, j] at B + k*ldb + j,
 * C[i, j] at C + i*ldc + j.  bias has N contiguous elements.  All four arrays
 * hold the same dtype.  Elements of C outside 0 <= j < N (the pitch padding)
 * are never written.
 *
 * Ownership: the caller owns every buffer; the library never frees, retains or
 * reads a pointer after the enqueued work completes.
 */
#ifndef TGEMM_H
#define TGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *tgemm_stream_t;   /* same handle as cudaStream_t; NULL = legacy default stream */

typedef enum { TGEMM_F16 = 0, TGEMM_BF16 = 1 } tgemm_dtype;

/*
 * GELU is the tanh form of "TileLang で GPU カーネル設計を解説" §4, written there
 * as a sigmoid: gelu(x) = x / (1 + exp(-1.5957691216 * (x + 0.044715 x^3))),
 * applied after the bias; evaluated in fp32 with CUDA's fast exponential.
 */
typedef enum {
    TGEMM_EPI_NONE = 0,       /* C = A.B                 */
    TGEMM_EPI_RELU = 1,       /* C = max(A.B, 0)         */
    TGEMM_EPI_BIAS = 2,       /* C = A.B + bias          */
    TGEMM_EPI_BIAS_RELU = 3,  /* C = max(A.B + bias, 0)  */
    TGEMM_EPI_GELU = 4,       /* C = gelu(A.B)           */
    TGEMM_EPI_BIAS_GELU = 5   /* C = gelu(A.B + bias)    */
} tgemm_epilogue;

typedef enum {
    TGEMM_OK = 0,
    TGEMM_ERR_INVALID_ARG = 1,        /* bad size, pitch, NULL pointer, dtype or epilogue   */
    TGEMM_ERR_ALIGNMENT = 2,          /* a base pointer is not 16-byte aligned               */
    TGEMM_ERR_UNSUPPORTED_DEVICE = 3, /* no CUDA device, or the current device is not CC 10.3 */
    TGEMM_ERR_ALIAS = 4,              /* C's byte range overlaps A, B or bias                */
    TGEMM_ERR_CUDA = 5,               /* a CUDA runtime/driver call or a launch failed       */
    TGEMM_ERR_TIMEOUT = 6,            /* a kernel gave up on a pipeline wait (device status) */
    TGEMM_ERR_SCRATCH_LIMIT = 7,      /* tgemm_run_noalloc: repacked operands exceed its fixed scratch */
    TGEMM_ERR_DEBUG_CHECK = 8,        /* debug build: a device-side bounds / alignment check failed
                                         and the access was skipped (device status) */
    TGEMM_ERR_CACHE = 9               /* a page number, length or start lies outside the cache; the
                                         rows that it stands for were left out (device status) */
} tgemm_status;

/*
 * tgemm_run — enqueue C = epi(A.B + bias) on `stream` (device pointers).
 *
 * Arguments: A [M x lda], B [K x ldb], bias [N] (may be NULL unless the
 * epilogue uses it: BIAS, BIAS_RELU, BIAS_GELU), C [M x ldc], all device
 * pointers in `dtype`.
 *
 * Errors are reported synchronously, before anything is enqueued, and leave C
 * untouched:
 *   M, N or K < 0; lda < K, ldb < N or ldc < N; a NULL A, B or C when the
 *   problem is not empty; a NULL bias with a BIAS epilogue; an unknown dtype or
 *   epilogue                                              -> TGEMM_ERR_INVALID_ARG
 *   a base pointer (A, B, C, bias) not 16-byte aligned    -> TGEMM_ERR_ALIGNMENT
 *   C's byte range overlapping A's, B's or bias's         -> TGEMM_ERR_ALIAS
 *   no device, or a current device other than CC 10.3    -> TGEMM_ERR_UNSUPPORTED_DEVICE
 *   a pointer the driver does not know as device memory   -> TGEMM_ERR_INVALID_ARG
 *   a failed CUDA call or launch                          -> TGEMM_ERR_CUDA
 *
 * Degenerate sizes: M == 0 or N == 0 enqueues nothing and returns TGEMM_OK;
 * K == 0 writes epi(bias) (the empty sum is 0).
 *
 * Any pitch >= the logical width is accepted.  When lda or ldb is not a
 * multiple of 8 elements (tensor-memory-access copies need 16-byte row
 * strides) the operand is first repacked on the GPU into a 16-byte-pitched
 * scratch buffer drawn stream-ordered from a library-owned memory pool and
 * returned to it on `stream`; when ldc is not a multiple of 8 the epilogue
 * stores C with plain masked stores instead of tensor-memory-access stores.
 * The library may read (never write) any element of the declared input
 * arrays, pitch padding included: a padded element only ever feeds outputs
 * outside C's M x N, which are not stored.
 *
 * Environment overrides of the work plan, for testing and tuning only (results
 * change at most by the split-K note below): TGEMM_FORCE_CFG (tile shape:
 * 256, 192, 128, 64, 256x2, 224x2, 128x2, or 256x4: two 256 x 256 CTA pairs
 * stacked in M that share B by cluster multicast), TGEMM_SPLIT_K (k ranges
 * for every tile), TGEMM_TAIL_SPLIT (the last partial wave's tiles: 0 = kept
 * whole, 1 = cut into column parts only), TGEMM_GROUP_M (row-blocks per
 * column sweep), TGEMM_NO_B3D (one copy per 64-column sub-tile of B).
 * TGEMM_TEST_STALL=1 (testing the failure path only) makes the GEMM kernel of
 * each call announce 16 bytes that never arrive for its first operand slot: its
 * operand wait runs out after 2 s, the kernel records TGEMM_ERR_TIMEOUT in the
 * device status word, drains and returns (C is left incomplete).
 * TGEMM_TRACE_MAX_GROUPS caps the persistent CTA groups in trace builds
 * (compiled with -DTGEMM_TRACE, never the product build) and is ignored
 * otherwise.
 *
 * Problems with too few output tiles to fill the GPU (few rows, e.g. decode
 * shapes) split the k loop of each tile across CTAs: fp32 partial sums go to
 * pool scratch and the last CTA to finish a tile region adds them in a fixed
 * order before the epilogue, so results are deterministic; they may differ
 * in the last bits from an unsplit run (different summation order).  The
 * arrival counters of those regions live in a small buffer the library keeps
 * for each stream it has launched such work on (8 bytes per region, at least
 * 4 KiB, drawn from its pool and kept until the process exits); calls on one
 * stream are ordered, so they share it safely.  Kernels are enqueued as
 * programmatic dependent launches: their set-up may overlap the end of the
 * stream's previous kernel, but they touch no global memory before that
 * kernel has completed, so stream order holds as for any launch.  Larger
 * problems whose tiles leave a last, partial wave cut those tiles the same
 * way (2-4 k ranges, each at least 16 k-blocks, when the pieces fit one wave;
 * same determinism, and those tiles may differ in the last bits from an
 * unsplit run), else into narrower column parts, which change no result bit.
 *
 * Asynchrony: returns once the work is enqueued; the caller synchronises.
 * Thread safety: safe to call from several host threads.
 */
tgemm_status tgemm_run(const void *A, const void *B, const void *bias, void *C,
                       int64_t M, int64_t N, int64_t K,
                       int64_t lda, int64_t ldb, int64_t ldc,
                       tgemm_dtype dtype, tgemm_epilogue epilogue, tgemm_stream_t stream);

/*
 * tgemm_run_ex — tgemm_run with either operand stored transposed (the
 * transpose_A / transpose_B options of T.gemm in "Writing high-performance
 * kernels in TileLang", "Écrivons un GEMM"; the column-major B of
 * "【CUDA】TileFusion").  The product is still C = epi(A.B + bias) with A
 * M x K and B K x N:
 *   transpose_a = 0: A[i, k] at A + i*lda + k   (stored [M, lda], lda >= K)
 *   transpose_a = 1: A[i, k] at A + k*lda + i   (stored [K, lda], lda >= M)
 *   transpose_b = 0: B[k, j] at B + k*ldb + j   (stored [K, ldb], ldb >= N)
 *   transpose_b = 1: B[k, j] at B + j*ldb + k   (stored [N, ldb], ldb >= K:
 *                    the [out_features, in_features] weight layout)
 * The tensor cores read either major directly; nothing is transposed in
 * memory.  Errors as tgemm_run (a transpose flag other than 0 or 1 ->
 * TGEMM_ERR_INVALID_ARG).
 */
tgemm_status tgemm_run_ex(const void *A, const void *B, const void *bias, void *C,
                          int64_t M, int64_t N, int64_t K,
                          int64_t lda, int64_t ldb, int64_t ldc,
                          tgemm_dtype dtype, tgemm_epilogue epilogue,
                          int transpose_a, int transpose_b, tgemm_stream_t stream);

/*
 * tgemm_run_host — the same operation on HOST buffers (pinned or pageable),
 * end to end: device buffers are drawn from the library's stream-ordered pool,
 * A, B and bias are copied host -> device on `stream`, tgemm_run is enqueued,
 * C is copied device -> host, and the buffers are returned to the pool.
 * The call returns after enqueueing; C_host is valid once `stream` has been
 * synchronised (with pageable memory the copies themselves may block).
 * Same arguments, pitches and errors as tgemm_run (no device-pointer check).
 */
tgemm_status tgemm_run_host(const void *A_host, const void *B_host, const void *bias_host,
                            void *C_host, int64_t M, int64_t N, int64_t K,
                            int64_t lda, int64_t ldb, int64_t ldc,
                            tgemm_dtype dtype, tgemm_epilogue epilogue, tgemm_stream_t stream);

/*
 * tgemm_run_noalloc — tgemm_run for callers that must not allocate GPU memory.
 * (No counterpart on the pages: this is a deployment variant of the same
 * operation.)
 *
 * Who needs it: code whose device memory is reserved up front by another
 * allocator (a framework's caching allocator that holds most of HBM, so a
 * library-side cudaMalloc/cudaMallocAsync can fail or fragment that reserve),
 * latency-bound loops that avoid allocation calls because they can block or
 * synchronise, and deployments that forbid any allocation after start-up.
 *
 * What differs from tgemm_run: nothing is allocated.  The only scratch this
 * operation needs — the repacked copy of A and/or B when lda or ldb is not a
 * multiple of 8 elements — lives in a fixed device array inside the library of
 * TGEMM_NOALLOC_SCRATCH_BYTES (64 MiB), which every GPU that loads the library
 * holds until the process exits.  Each repacked operand takes
 * rows * round_up(width, 8) * 2 bytes, rounded up to 256 bytes; if the
 * operands that need repacking do not fit together, the call returns
 * TGEMM_ERR_SCRATCH_LIMIT before enqueueing anything.  Operands whose pitch is
 * already a multiple of 8 use no scratch at all.
 *
 * Sharing: every call, on every stream and host thread, uses the same array,
 * so two calls that may overlap on the GPU race on it; order them (one
 * stream, or events).  The array keeps the previous call's contents; nothing
 * in it needs to start at zero, because each call writes every scratch
 * element it reads before reading it.
 *
 * Set-up: the first call on each device (with that device current) looks up
 * the device address of the array once; make that first call before any
 * stream capture.
 *
 * Arguments, layout and the other error codes are those of tgemm_run.
 * Results: this variant never splits the k loop (the fp32 partial sums would
 * need scratch), while tgemm_run splits it for problems with few output tiles
 * and may split the tiles of a last, partial wave.  The two therefore agree
 * bit for bit wherever tgemm_run's plan has no k split (tgemm_plan reports
 * split_k == 1) and whenever every partial sum is exact (small-integer
 * inputs); otherwise both are within the same error bound of the exact
 * result and may differ in the last bits.
 */
#define TGEMM_NOALLOC_SCRATCH_BYTES (64ull << 20)
tgemm_status tgemm_run_noalloc(const void *A, const void *B, const void *bias, void *C,
                               int64_t M, int64_t N, int64_t K,
                               int64_t lda, int64_t ldb, int64_t ldc,
                               tgemm_dtype dtype, tgemm_epilogue epilogue, tgemm_stream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char *tgemm_status_string(tgemm_status status);

/*
 * tgemm_last_device_status — read and clear the device-side status word of the
 * current device.  Kernels bound every pipeline wait by a time limit; a wait
 * that runs out records TGEMM_ERR_TIMEOUT here and the kernel returns early
 * (its output is then invalid).  In the debug build a failed device-side check
 * records TGEMM_ERR_DEBUG_CHECK, and the first error since the last call is
 * kept (the release build keeps the last).  Synchronises the device.  Returns TGEMM_OK when no kernel has reported an
 * error since the last call.
 */
tgemm_status tgemm_last_device_status(void);

/*
 * tgemm_debug_last_check — the debug build (libtgemm_debug.so, compiled with
 * -DTGEMM_DEBUG; the Python binding loads it when TGEMM_DEBUG=1 is set): the
 * id of the first device-side check that failed since the last call, then
 * cleared; 0 when none failed.  The checks guard the error classes the
 * TileLang tutorial names for hand-written kernels: 1 / 2 a TMA load of A /
 * B whose innermost coordinate is not 16-byte aligned, 3 a TMA store of C
 * starting at a negative, unaligned or out-of-range coordinate, 4 a plain
 * store of C outside its (M - 1) * ldc + N elements, 5 a split-K partial
 * outside its scratch, 6 an arrival counter outside its buffer, 7 an
 * attention output store outside O, 8 a repack store outside its
 * destination, 9 a row of the paged cache written outside its pool, 10 an
 * output of tgemm_attention_decode, tgemm_kv_evict, tgemm_kv_bounds or
 * tgemm_kv_select outside its array, 11 a part or score outside the workspace,
 * 12 a rotated row or its gradient outside its array.  The failing access is skipped (nothing traps); a skipped
 * copy leaves its pipeline slot incomplete, which the bounded waits end.
 * Synchronises the device.  Returns -1 in the release build, which compiles
 * no checks.  Testing only: TGEMM_DEBUG_PLANT=c_store makes the debug build's
 * bound for C one row short, so that check 4 fires on C's last row (whose
 * stores are then skipped).
 */
int tgemm_debug_last_check(void);

/* Library version, e.g. 0x000100 for 0.1.0. */
int tgemm_version(void);

/*
 * tgemm_attention_fwd — enqueue the attention forward pass (the output of
 * FlashAttention, "TileLang で GPU カーネル設計を解説" §6) on `stream`:
 *
 *   O[b, i, h, :] = sum_j softmax_j(scale * Q[b, i, h, :] . K[b, j, h, :]) V[b, j, h, :],
 *   scale = 1 / sqrt(dim),
 *
 * over all keys j < seq, or only j <= i when causal = 1.
 *
 * Arguments: Q, K, V, O device pointers in `dtype` (fp16 or bf16), each a
 * dense [batch, seq, heads, dim] array (dim contiguous, then heads, then seq,
 * then batch), 16-byte aligned; O must not overlap Q, K or V.  dim must be 64.
 * Ownership stays with the caller; the call only reads Q, K, V and writes O.
 *
 * Arithmetic: scores and P.V products accumulate in fp32; the softmax runs
 * blockwise over 128 keys at a time with a running maximum and sum (the
 * online softmax), P is rounded to `dtype` before it multiplies V, and each
 * output row is divided by the fp32 sum of the unrounded P and rounded once
 * to `dtype` (round-to-nearest-even).
 *
 * Returns TGEMM_ERR_INVALID_ARG (negative sizes, dim != 64, causal not 0/1,
 * bad dtype, batch or heads above 65535, a NULL or host pointer for a
 * non-empty problem), TGEMM_ERR_ALIGNMENT, TGEMM_ERR_ALIAS,
 * TGEMM_ERR_UNSUPPORTED_DEVICE, TGEMM_ERR_CUDA; TGEMM_OK once enqueued.
 * An empty problem (batch, seq or heads 0) enqueues nothing.
 */
tgemm_status tgemm_attention_fwd(const void *Q, const void *K, const void *V, void *O,
                                 int64_t batch, int64_t seq, int64_t heads, int64_t dim,
                                 int causal, tgemm_dtype dtype, tgemm_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The paged key-value cache: what attention needs when tokens come one at a
 * time.  (No counterpart on the pages, which stop at whole sequences.)
 *
 * Keys and values live in two pools of rows.  A row holds the `dim` elements of
 * one head at one position; position pos of a sequence lies on page
 * list[pos / page_size] of the pools, at slot pos % page_size, where list is the
 * sequence's row of a page table:
 *   row(page, slot, head) = base + page * page_stride + slot * slot_stride
 *                                + head * head_stride            (elements)
 * so that [page, slot, head, dim] and [page, head, slot, dim] pools, and pools
 * that hold keys and values side by side, are all described by strides.  K and
 * V share the strides.  Elements are fp16 or bf16 (the calls' dtype), or, with
 * e4m3 = 1, e4m3 with one fp32 scale per row and pool: value = scale * element,
 * scale >= 0.
 *
 * Limits: dim a multiple of 8 (e4m3: 16), at most 256; page_size 1 .. 2^20;
 * bases 16-byte aligned and strides multiples of 16 bytes; rows may not
 * overlap.
 */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;                                           /* e4m3 = 1 only */
    int64_t pages;
    int64_t page_stride, slot_stride, head_stride;                      /* elements      */
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;    /* floats        */
    int32_t page_size, heads, dim, e4m3;
} tgemm_kv_cache;

/*
 * Sequences that share a cache.
 *   pages    int32 [batch, pages_stride], device: each sequence's page list, of
 *            pages_width entries at most; entries past a sequence's length are
 *            not read.  pages_width * page_size is at most 2^30.
 *   lengths  int32 [batch], device: positions each sequence holds.
 * batch is at most 65535.
 */
typedef struct {
    const int32_t *pages;
    const int32_t *lengths;
    int64_t pages_width, pages_stride, batch;
} tgemm_kv_sequences;

/* Accumulated attention weights, fp32 [batch, heads, width], device (data NULL: none). */
typedef struct {
    float *data;
    int64_t width, batch_stride, head_stride;
} tgemm_kv_weights;

/*
 * Common to the calls on the cache below.
 *
 * Page numbers, lengths and starts are on the device, so the kernels check
 * them: one that lies outside the pool or the table (a negative length too) is
 * recorded as TGEMM_ERR_CACHE in the device status word
 * (tgemm_last_device_status), and the rows that it stands for are left out;
 * nothing outside the arrays is read or written.
 *
 * Errors that the host sees are returned before anything is enqueued:
 * TGEMM_ERR_INVALID_ARG (sizes, strides, dtype, a NULL or host pointer),
 * TGEMM_ERR_ALIGNMENT, TGEMM_ERR_ALIAS, TGEMM_ERR_UNSUPPORTED_DEVICE,
 * TGEMM_ERR_CUDA.  The argument structures are read during the call only.
 * Nothing is allocated and the host does not read device memory, so the calls
 * can be captured into a graph, which then follows the lengths and pages that
 * it finds at each replay.
 */

/*
 * tgemm_kv_append — write the newest tokens' rows.  K and V are
 * [tokens, heads, dim] (strides in elements, multiples of 8).  Sequence b
 * brings the tokens starts[b] .. starts[b + 1] - 1 (starts: int32 [batch + 1],
 * ascending, device); with starts = NULL each brings one (tokens = batch).
 * lengths[b] counts them already: the last of them goes to position
 * lengths[b] - 1.  Tokens outside starts[0] .. starts[batch] - 1 are left out.
 * An e4m3 row's scale is max |x| / 448 (1 for a row of zeros) and its elements
 * x / scale, rounded to nearest even.  A NaN stays one and does not count in its
 * row's maximum; an infinity makes the scale infinite, so that its row reads as
 * NaN.  With weights, those of the new positions are set to 0.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    tgemm_kv_sequences seq;
    tgemm_kv_weights weights;
    const void *K, *V;
    const int32_t *starts;
    int64_t tokens, token_stride, head_stride;
    int64_t dtype;                                  /* tgemm_dtype of K and V */
} tgemm_kv_append_args;
tgemm_status tgemm_kv_append(const tgemm_kv_append_args *args, tgemm_stream_t stream);

/*
 * tgemm_attention_decode — attention of one new token per sequence over its
 * cache.  Q and O are [batch, q_heads, dim] with strides (multiples of 8
 * elements); query head h reads the keys of head h / (q_heads / heads).
 *
 *   O[b, h] = sum_j p_j V[b, j],  p = softmax of s_j over max(0, n - window) <= j < n,  n = lengths[b],
 *   s_j = scale * Q[b, h] . K[b, j], passed through cap * tanh(s / cap) when cap > 0;
 *
 * window = 0: all positions.  batch * q_heads * (what the page lists can hold)
 * is at most 2^42.  A sequence of length 0 gets zeros.  Rows past n,
 * NaN and infinity among them, have no influence.  With weights,
 * weights[b, g, j] grows by the sum of p_j over the query heads of group g.
 *
 * Arithmetic: products of 16-bit values (e4m3 elements are widened exactly)
 * accumulated in fp32; softmax in fp32 with a running maximum, each weight
 * multiplying V as the sum of two 16-bit values (off by at most 2^-16 of itself
 * with bf16 keys and values, 2^-21 with fp16 and e4m3); each output rounded once
 * to dtype.  With fp16 keys and values weights below 2^-32 of the largest are
 * lost; with e4m3, where weight times value scale is below 2^-31 of the largest
 * such product of a row that is not all zeros.  Values near 2^119 and above may
 * overflow fp32 before the sum of the weights is divided out.
 *
 * workspace: device memory of tgemm_attention_decode_workspace() bytes,
 * 16-byte aligned, that held zeros before its first use; the call leaves it fit
 * for the next.  Calls that may overlap on the GPU need one each.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    tgemm_kv_sequences seq;
    tgemm_kv_weights weights;
    const void *Q;
    void *O;
    int64_t q_heads, q_batch_stride, q_head_stride, o_batch_stride, o_head_stride;
    int64_t window;
    double scale, cap;
    void *workspace;
    int64_t workspace_bytes;
    int64_t dtype;                                  /* tgemm_dtype of Q and O */
} tgemm_attention_decode_args;
tgemm_status tgemm_attention_decode(const tgemm_attention_decode_args *args, tgemm_stream_t stream);

/*
 * Bytes of workspace that tgemm_attention_decode needs for up to `batch`
 * sequences of up to `positions` positions (pages_width * page_size).  Host
 * logic only.
 */
tgemm_status tgemm_attention_decode_workspace(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim,
                                              int64_t positions, int with_weights, int64_t *bytes);

/*
 * tgemm_kv_evict — bring sequences back to at most `keep` positions.  Of n =
 * lengths[b] positions each head keeps k = min(n, keep): the last
 * r = min(recent, k), and of the n - r before them the k - r of largest weight
 * (ties to the lowest position, NaN below every number).  Their rows go, in
 * order, to positions 0 .. k - 1 of the page lists of `to_seq` in the cache
 * `to`, with scales and weights.  `to` may describe the same pools as `from` as
 * long as the pages written are not among those read (pages may be shared by
 * sequences: nothing of `from` changes).  to_seq.lengths is not used.  Outputs
 * besides the rows:
 *   kept        int32 [batch, heads, keep]: the positions kept, ascending, -1 from k on
 *   to_lengths  int32 [batch]: k
 *   to_weights  fp32 [batch, heads, width >= keep]: the weights kept, 0 from k to keep - 1
 */
typedef struct {
    const tgemm_kv_cache *from;
    tgemm_kv_sequences seq;
    tgemm_kv_weights weights;
    const tgemm_kv_cache *to;
    tgemm_kv_sequences to_seq;
    tgemm_kv_weights to_weights;
    int32_t *kept;
    int32_t *to_lengths;
    int64_t keep, recent;
} tgemm_kv_evict_args;
tgemm_status tgemm_kv_evict(const tgemm_kv_evict_args *args, tgemm_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Sparse attention: pages that a cheap score selects.
 *
 * For each page and key head, each channel's least and largest key in 8 bits:
 *   bounds  int8 [pages, heads, 2, dim], contiguous, 16-byte aligned: lo, then hi
 *   scale   fp32 [pages, heads]: s, the least power of two (2^-100 at least)
 *           such that no key of the page exceeds 127 s in magnitude
 *   lo = floor(min k / s), hi = ceil(max k / s), so that s lo <= k <= s hi.
 * The keys of an e4m3 cache are the fp32 products scale * element.  A NaN counts
 * as not there, an infinity as the largest finite number.  dim is a multiple of 16.
 */
typedef struct {
    int8_t *bounds;
    float *scale;
} tgemm_kv_page_bounds;

/*
 * tgemm_kv_bounds — the bounds of the pages that the newest tokens complete.
 * Sequence b has brought starts[b + 1] - starts[b] tokens (starts: int32 [batch
 * + 1], device; NULL: one each), which lengths[b] counts already: the pages
 * whose last position is among them are read whole and their bounds written.
 * Call it after tgemm_kv_append.  A page that is not full has no bounds.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    const tgemm_kv_page_bounds *bounds;
    tgemm_kv_sequences seq;
    const int32_t *starts;
    int64_t dtype;                                  /* of the keys of a 16-bit cache */
} tgemm_kv_bounds_args;
tgemm_status tgemm_kv_bounds(const tgemm_kv_bounds_args *args, tgemm_stream_t stream);

/*
 * tgemm_kv_select — of each sequence's pages, each key head keeps at most `keep`:
 * the first `first`, the last `recent` (1 at least: the last page may not be
 * full), and of those between them the ones of largest score (ties to the lowest
 * position).  With z the query of a head (Q [batch, q_heads, dim], as in
 * tgemm_attention_decode) in whole numbers of a power of two t, found as s is
 * above (rounded to nearest even), a page's score is the largest over the head's
 * group of
 *     t s sum_d max(z_d lo_d, z_d hi_d)   (z_d lo_d for z_d < 0, z_d hi_d for z_d > 0)
 * in fp32, which is exact from 2^-104 to the end of fp32's range.  Written, for
 * tgemm_attention_decode_lists:
 *   to_pages    int32 [batch, heads, keep]: page numbers in order of position, -1 past them
 *   to_lengths  int32 [batch]: positions on them
 * first + recent <= keep; at most 2^17 pages in a list and 64 query heads on a
 * key head.  A page number outside the cache is recorded and scores lowest.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    const tgemm_kv_page_bounds *bounds;
    tgemm_kv_sequences seq;
    const void *Q;
    int64_t q_heads, q_batch_stride, q_head_stride;
    int32_t *to_pages;
    int32_t *to_lengths;
    int64_t to_batch_stride, to_head_stride;
    int64_t keep, first, recent;
    int64_t dtype;                                  /* tgemm_dtype of Q */
} tgemm_kv_select_args;
tgemm_status tgemm_kv_select(const tgemm_kv_select_args *args, tgemm_stream_t stream);

/*
 * tgemm_attention_decode_lists — tgemm_attention_decode with a page list for each
 * key head: seq.pages is [batch, heads, pages_width] with strides seq.pages_stride
 * and pages_head_stride (at least pages_width; 0: the heads share a list).
 * Positions, the window's and the weights' too, are those of the lists.
 */
tgemm_status tgemm_attention_decode_lists(const tgemm_attention_decode_args *args, int64_t pages_head_stride,
                                          tgemm_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The pages as a resource.  uses, int32 [pages] on the device, counts the
 * sequences that hold each page; 0: free.  A list that a call below writes is not
 * one that the same call reads, except where it says so.  New pages are the
 * lowest free ones, in the order of the sequences.  What cannot be done (no page
 * left, a list without room, a bad length, parent or page number) is recorded as
 * TGEMM_ERR_CACHE and left out.  The sums of 1024 sequences' list widths stay
 * below 2^31, pages and page_size * heads at most 2^30.
 */

/*
 * tgemm_kv_grow — room for new tokens: lengths[b] grows by tokens[b] (int32
 * [batch], device; NULL: one each), and the list by the pages that this takes.
 * From the first sequence on whose pages are not there, those that need any stay
 * as they are.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    int32_t *uses;
    int32_t *pages;                                 /* [batch, pages_stride] */
    int32_t *lengths;
    int64_t pages_width, pages_stride, batch;
    const int32_t *tokens;
} tgemm_kv_grow_args;
tgemm_status tgemm_kv_grow(const tgemm_kv_grow_args *args, tgemm_stream_t stream);

/*
 * tgemm_kv_fork — child c takes over the positions of sequence parents[c] of
 * `seq` (int32 [children], device; -1: none, the child is empty): full pages are
 * shared, the rows of a last, partly filled page are copied to a page of the
 * child's own.  Where no page is left a child has the full pages alone.  The
 * children's lists and lengths (whose old contents are lost, not freed) may be
 * other rows of the parents' arrays, as long as no child is a parent.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    int32_t *uses;
    tgemm_kv_sequences seq;
    const int32_t *parents;
    int32_t *to_pages;                              /* [children, to_stride] */
    int32_t *to_lengths;
    int64_t to_width, to_stride, children;
} tgemm_kv_fork_args;
tgemm_status tgemm_kv_fork(const tgemm_kv_fork_args *args, tgemm_stream_t stream);

/*
 * tgemm_kv_free — the sequences give their pages back: each is held once less, and lengths become 0 (a length that
 * the list cannot hold, and its sequence, stay as they are).
 */
typedef struct {
    const tgemm_kv_cache *cache;
    int32_t *uses;
    const int32_t *pages;                           /* [batch, pages_stride] */
    int32_t *lengths;
    int64_t pages_width, pages_stride, batch;
} tgemm_kv_free_args;
tgemm_status tgemm_kv_free(const tgemm_kv_free_args *args, tgemm_stream_t stream);

/*
 * tgemm_kv_compact — of the pages in use, those numbered n = (their number) and
 * above move, in order, to the free ones below n, in order, with scales and, if
 * given, bounds.  `seq` has all sequences that hold pages.  Written:
 *   to_pages  int32 [batch, to_stride]: the lists with the new numbers (entries past a length are left)
 *   to_uses   int32 [pages]: the counts
 *   in_use    int32 [1]: n; from page n on the pool is free
 * to_pages may be seq.pages (with its stride), to_uses may be uses.  workspace:
 * device memory of tgemm_kv_compact_workspace() bytes, 16-byte aligned; calls
 * that may overlap on the GPU need one each.  Of a length past what its list
 * holds all of the list is translated, as pages move all the same.
 */
typedef struct {
    const tgemm_kv_cache *cache;
    const tgemm_kv_page_bounds *bounds;             /* NULL: none */
    const int32_t *uses;
    tgemm_kv_sequences seq;
    int32_t *to_pages;
    int64_t to_width, to_stride;
    int32_t *to_uses;
    int32_t *in_use;
    void *workspace;
    int64_t workspace_bytes;
} tgemm_kv_compact_args;
tgemm_status tgemm_kv_compact(const tgemm_kv_compact_args *args, tgemm_stream_t stream);

/* Bytes of workspace that tgemm_kv_compact needs for a cache of `pages` pages.  Host logic only. */
tgemm_status tgemm_kv_compact_workspace(int64_t pages, int64_t *bytes);

/*
 * ---------------------------------------------------------------------------
 * Norms of queries and keys for each head, with the position rotation in the
 * same pass.
 */

/* Rows of heads, [tokens, heads, dim]: base and strides (elements, multiples of 8; bases 16-byte aligned). */
typedef struct {
    void *data;
    int64_t token_stride, head_stride;
} tgemm_rows;

/*
 * A rotation of the first 2 * pairs elements of a row, host memory:
 *   turns        uint64 [pairs]: how far a pair turns per position, as a fraction
 *                of 2^64 of a whole turn (frequency / (2 pi) * 2^64)
 *   axes         int32 [pairs]: whose positions count (NULL: all 0)
 *   interleaved  0: pair i is elements i and i + pairs (pairs a multiple of 4);
 *                1: elements 2 i and 2 i + 1
 */
typedef struct {
    const uint64_t *turns;
    const int32_t *axes;
    int64_t pairs, interleaved;
} tgemm_rotary;

/*
 * tgemm_qk_norm_rope — for each row x of the queries and keys of a token
 *
 *   y = R(x * r * weight),   r = 1 / sqrt(mean x^2 + eps)
 *
 * (norm = 0: y = R(x), no weights), R turning pair i by the angle
 * (positions[axes[i], token] + shift) * frequency_i; rotary NULL: no rotation.
 * Weights have dim contiguous elements of `dtype`, or fp32 with weight_f32 = 1;
 * NULL: ones.  positions is int32 [axes, tokens], device, any values
 * (axis_stride 0: the axes share them), axes at most 32; position * frequency
 * keeps 2^-31 of a turn whatever they are, the rest is fp32, rounded once (a row
 * whose sum of squares passes fp32's range becomes zeros).  eps lies in fp32's
 * range; with 0 a row whose mean square fp32 rounds to 0 is not finite.  dim is a multiple of
 * 8, at most 256.  q_heads or k_heads may be 0.  q_out and k_out may be q and k
 * themselves (the same strides), and may lie side by side with others in one
 * array; they overlap nothing else.
 */
typedef struct {
    tgemm_rows q, k, q_out, k_out;
    const void *q_weight, *k_weight;
    const int32_t *positions;
    int64_t axis_stride, axes, tokens, q_heads, k_heads, dim, shift;
    const tgemm_rotary *rotary;
    int64_t weight_f32, norm;
    double eps;
    int64_t dtype;
} tgemm_qk_norm_rope_args;
tgemm_status tgemm_qk_norm_rope(const tgemm_qk_norm_rope_args *args, tgemm_stream_t stream);

/*
 * tgemm_qk_norm_rope_backward — the gradients of tgemm_qk_norm_rope: of q and k,
 * written to forward.q_out and forward.k_out (which may be q and k, or q_grad and
 * k_grad, themselves), from those of what it wrote, q_grad and k_grad; and of the
 * weights, fp32 [dim], written, not added (NULL: not wanted; they need norm = 1
 * and the workspace).  Sums are fp32 in a fixed order: results are deterministic.
 * With norm = 0 q and k are not read.  Rows whose sums pass fp32's range have
 * gradients that are not finite.  workspace: device memory of
 * tgemm_qk_norm_rope_backward_workspace() bytes, 16-byte aligned, that held zeros
 * before its first use; the call leaves it fit for the next.  Calls that may
 * overlap on the GPU need one each.
 */
typedef struct {
    tgemm_qk_norm_rope_args forward;
    tgemm_rows q_grad, k_grad;
    float *q_weight_grad, *k_weight_grad;
    void *workspace;
    int64_t workspace_bytes;
} tgemm_qk_norm_rope_backward_args;
tgemm_status tgemm_qk_norm_rope_backward(const tgemm_qk_norm_rope_backward_args *args, tgemm_stream_t stream);

/* Bytes of workspace that tgemm_qk_norm_rope_backward needs.  Host logic only. */
tgemm_status tgemm_qk_norm_rope_backward_workspace(int64_t dim, int64_t *bytes);

/*
 * tgemm_plan — the work plan tgemm_run (and tgemm_run_ex / tgemm_run_host per
 * chunk) uses for an M x N x K problem on a GPU with num_sms SMs.  Host logic
 * only: no device is touched, so it also answers on a machine without a GPU.
 * The transposed layouts do not change the plan; tgemm_run_noalloc uses it
 * with split_k forced to 1.
 *
 * out (caller-owned, 10 int32 entries):
 *   [0] tile width BN (columns)      [1] CTAs per tile (1; 2 for a pair: 256 rows;
 *                                        4 for two pairs sharing B: 512 rows)
 *   [2] shared-memory ring stages    [3] tiles = ceil(M / (128 * [1])) * ceil(N / BN)
 *   [4] persistent CTA groups launched (CTAs = [4] * [1])
 *   [5] split_k (1: no k split)      [6] first tile split in k (tiles from here on)
 *   [7] first narrow tile            [8] column parts of each narrow tile (1: none);
 *                                        tiles [7] .. [6]-1 are cut into [8] parts
 *   [9] work units of the persistent loop
 *
 * The tile-shape rule and the plan are heuristics: they may change between
 * versions without changing any result beyond the split-K note of tgemm_run.
 * Returns TGEMM_ERR_INVALID_ARG if out is NULL, num_sms < 2, or a size is
 * below 1 or above INT32_MAX; TGEMM_OK otherwise.
 */
tgemm_status tgemm_plan(int64_t M, int64_t N, int64_t K, int num_sms, int32_t *out);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_H */
