/*
 * qgemv: batch-1 GEMV with block-quantised weights dequantised on the fly, for GB300
 * (sm_103a).
 *
 *     y[n] = sum_k x[k] * dequant(W)[n, k],   n < N, k < K        (M = 1, alpha = 1, beta = 0)
 *
 * The operation is the GEMV of "Writing a high performant GEMV + dequant for Metal"
 * (section "What is a GEMV": y = alpha x.W^T + beta C with x:(1,K), W:(M,K), alpha = 1,
 * beta = 0; that page's M is N here) and of the Mojo "fp4_gemv" page (out = x @ dequant(W)^T
 * at M = 1).  Weights stay in their packed block format in device memory; every kernel
 * streams the packed bytes once, decodes them in registers and accumulates in fp32.
 *
 * Conventions for every entry point:
 *  - Pointers named x, W, y, codes, scales, mins are DEVICE pointers owned by the caller.
 *    The library never frees, keeps or retains them past the call's stream work.
 *  - Calls are asynchronous on `stream`; nothing is allocated and nothing synchronises
 *    inside qgemv_run / qgemv_unpack.  Results are ready when the stream's work is done.
 *  - Errors are reported only through the returned status; arguments are validated before
 *    anything is launched, so an error status means no kernel was enqueued (except
 *    QGEMV_ERR_CUDA, which means the launch itself failed).
 *  - A handle may be used from one host thread at a time.
 */
#ifndef QGEMV_H_
#define QGEMV_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Weight formats.  Byte layouts (offsets inside one block, fp16 little-endian):
 *  QGEMV_Q4_K  256 weights / 144 B: d@0, dmin@2, 12 B packed 6-bit scales+mins@4,
 *              qs[128]@16.  w_i = d*s_g*q_i - dmin*m_g, g = i/32 (Metal GEMV page,
 *              sections "What is a weight block?" and "Compute").  x fp16.
 *  QGEMV_NVFP4 W4A16 (Mojo fp4_gemv page, "Structure"): E2M1 nibbles [N, K/2] (low nibble
 *              = even k) immediately followed, in the SAME buffer, by E4M3 scales
 *              [N, K/16]; w = e2m1 * |e4m3 scale of its 16-element block|.  x bf16.
 *  QGEMV_TQ1_0 256 weights / 54 B: qs[48]@0 (5 base-3 digits per byte), qh[4]@48
 *              (4 digits per byte), d@52; digit n of byte b = floor(3^(n+1) b/256) -
 *              3 floor(3^n b/256); w = d*(t-1) ("metal: TQ1_0 kernel performance",
 *              sections 1, 2 and "Not applicable").  x fp16.
 *  QGEMV_Q5_K  256 weights / 176 B: d@0, dmin@2, scales[12]@4, qh[32]@16, qs[128]@48.
 *  QGEMV_Q6_K  256 weights / 210 B: ql[128]@0, qh[64]@128, int8 scales[16]@192, d@208.
 *  QGEMV_Q8_0   32 weights /  34 B: d@0, int8 qs[32]@2.
 *  (Q5_K, Q6_K and Q8_0 are named on the Metal GEMV page, section "UD-Q4_K_XL"; their
 *  standard ggml layouts are used.)  x fp16 for all of them. */
typedef enum {
  QGEMV_Q4_K = 0,
  QGEMV_NVFP4 = 1,
  QGEMV_TQ1_0 = 2,
  QGEMV_Q5_K = 3,
  QGEMV_Q6_K = 4,
  QGEMV_Q8_0 = 5
} qgemv_format_t;

typedef enum {
  QGEMV_OK = 0,
  QGEMV_ERR_INVALID_ARG = 1,        /* null pointer / handle, bad option value */
  QGEMV_ERR_UNSUPPORTED_FORMAT = 2, /* format id not in qgemv_format_t */
  QGEMV_ERR_BAD_SHAPE = 3,          /* N < 1, K < 1, K not a multiple of the block length */
  QGEMV_ERR_MISALIGNED = 4,         /* x, W or y not 16-byte aligned */
  QGEMV_ERR_CUDA = 5,               /* a CUDA runtime call or kernel launch failed */
  QGEMV_ERR_TIMEOUT = 6,            /* a kernel gave up on a bounded wait (see check_error) */
  QGEMV_ERR_OOM = 7,                /* qgemv_create could not allocate its workspace */
  QGEMV_ERR_NO_DEVICE = 8,          /* no usable CUDA device / not an sm_103 device */
  QGEMV_ERR_TOO_LARGE = 9,          /* shape needs more than qgemv_run_noalloc's fixed scratch */
  QGEMV_ERR_BAD_INDEX = 10          /* a kernel met an index out of range (see check_error) */
} qgemv_status_t;

typedef struct qgemv_handle_s* qgemv_handle_t;

/* Create a handle on CUDA device `device` (made current for the call).  Queries the SM
 * count and L2 size and allocates the handle's device memory: a 4-byte error word, a 16 MiB
 * workspace for split-K column sums and 4 KiB of per-range counters (zeroed here; every
 * launch leaves them at zero).  *h receives the handle.  Returns QGEMV_ERR_NO_DEVICE when
 * the device is missing or is not compute capability 10.3, QGEMV_ERR_OOM when an allocation
 * fails. */
qgemv_status_t qgemv_create(qgemv_handle_t* h, int device);

/* Free the handle's device memory and the handle.  Waits for nothing: the caller must
 * make sure no work using the handle is still pending.  NULL is accepted. */
qgemv_status_t qgemv_destroy(qgemv_handle_t h);

/* y = x . dequant(W)^T  (overwrites y).
 *   x        device, K elements: fp16 bits (bf16 for QGEMV_NVFP4), 16-byte aligned.
 *   packed_W device, qgemv_packed_bytes(fmt, N, K) bytes, rows contiguous, 16-byte aligned.
 *   y        device, N fp32 values, 16-byte aligned; must not overlap x or packed_W.
 *   N >= 1; K >= 1 and a multiple of 256 (Q4_K, Q5_K, Q6_K, TQ1_0), 32 (Q8_0) or 16 (NVFP4).
 * The call is asynchronous on `stream` (0 = legacy default stream), allocates nothing and
 * does not synchronise.  It may use the handle's workspace, so calls on one handle must not
 * run at the same time on the GPU: calls ordered on one stream are fine; concurrent streams
 * need one handle each.  Results are deterministic: the same inputs and shape give
 * bitwise-identical y on every call (every sum is taken in a fixed order; the one atomic,
 * a per-range arrival count, only picks which CTA adds the column sums). */
qgemv_status_t qgemv_run(qgemv_handle_t h, qgemv_format_t fmt, const void* x, const void* packed_W,
                         int64_t N, int64_t K, float* y, cudaStream_t stream);

/* Debug unpack for bit-exact checks: for every weight (n, k)
 *     dequant(W)[n, k] = scales[n, k/G] * codes[n, k] - mins[n, k/G]      (exactly, in fp32)
 * with G = qgemv_group_size(fmt) and
 *   Q4_K, Q5_K: codes = q (0..15 / 0..31), scales = d*s_g, mins = dmin*m_g   (G = 32)
 *   Q6_K:       codes = q-32 (-32..31),    scales = d*sc,    mins = 0        (G = 16)
 *   Q8_0:       codes = int8 q,            scales = d,       mins = 0        (G = 32)
 *   TQ1_0:      codes = t-1 (-1..1),       scales = d,       mins = 0        (G = 256)
 *   NVFP4:      codes = 2*e2m1 (-12..12),  scales = |e4m3|/2, mins = 0       (G = 16)
 * All scales and mins are exact in fp32.  codes: device int8 [N, K]; scales: device fp32
 * [N, K/G]; mins: device fp32 [N, K/G] or NULL.  Same validation as qgemv_run (codes,
 * scales, mins need no 16-byte alignment).  Asynchronous on `stream`. */
qgemv_status_t qgemv_unpack(qgemv_handle_t h, qgemv_format_t fmt, const void* packed_W, int64_t N,
                            int64_t K, int8_t* codes, float* scales, float* mins, cudaStream_t stream);

/* Synchronise `stream`, then read and clear the handle's device error word.  Returns
 * QGEMV_ERR_TIMEOUT if any kernel since the last check gave up on a bounded wait (its y
 * is then undefined), QGEMV_ERR_BAD_INDEX if one met an index out of range in device memory
 * (a page, slot, position, length or adapter; what it did instead is said at its entry
 * point), QGEMV_ERR_CUDA if the stream reported an error, else QGEMV_OK. */
qgemv_status_t qgemv_check_error(qgemv_handle_t h, cudaStream_t stream);

/* Static description of a status code (never NULL). */
const char* qgemv_status_string(qgemv_status_t status);

/* Bytes of a packed N x K matrix in `fmt` (0 for an unknown format or a bad shape). */
size_t qgemv_packed_bytes(qgemv_format_t fmt, int64_t N, int64_t K);

/* Group length G of qgemv_unpack's scales for `fmt` (0 for an unknown format). */
int qgemv_group_size(qgemv_format_t fmt);

/* Tuning and test options (per handle).  Values are validated; bad ones give
 * QGEMV_ERR_INVALID_ARG and change nothing.
 *   QGEMV_OPT_FORCE_PATH      0 auto, 1 the cp.async streaming kernels (falls back to 0
 *                             when the shape does not meet their alignment rule) and, in
 *                             qgemv_run_batch, the batch kernel for every M >= 2 it takes
 *                             (whatever N), 2 the plain warp-per-row kernels.
 *   QGEMV_OPT_RING_DEPTH      0 auto, else 2..8: copy stages per warp of the streaming
 *                             kernel (2, 3 or 4 are used, larger values mean 4; fewer
 *                             if they do not fit in shared memory).
 *   QGEMV_OPT_ROWS_PER_STAGE  0 auto, else 1..8 rows per stage (1, 2 or 4 are used).
 *   QGEMV_OPT_SPIN_LIMIT_NS   bound, in ns, of every spin-wait on a barrier in the kernels
 *                             (default 1e9); 0 makes such a wait give up at once.  (The
 *                             streaming kernel waits for its own copies with
 *                             cp.async.wait_group, which the hardware completes.)
 *   QGEMV_OPT_PDL             1 launches the streaming kernels with programmatic dependent
 *                             launch: they may start while the previous kernel on the stream
 *                             is still running, and they request their first weight stages
 *                             before waiting for it; activations are read only after it
 *                             completes.  packed_W must therefore not be written by the kernel
 *                             launched just before.  0 (default) launches them normally.
 *   QGEMV_OPT_TEST_STALL      test hook, default 0.  1 makes warp 0 of the first CTA of every
 *                             streaming launch also wait on a barrier that nothing completes,
 *                             bounded by the spin limit, so the timeout path (error word,
 *                             draining of in-flight copies, QGEMV_ERR_TIMEOUT from
 *                             qgemv_check_error) can be exercised without hanging a GPU; in
 *                             qgemv_run_gemm's tensor-core kernel, the first CTA's
 *                             dequantising threads withhold their arrival for its first stage,
 *                             so its MMA, copy and dequantising waits all run out.
 *   QGEMV_OPT_CTAS_PER_SM     streaming kernel CTAs per SM, 1 or 2 (default 2, used when
 *                             a row needs at most 8 warps); with 1, each CTA takes about half
 *                             an SM, so the next kernel of a programmatic-dependent-launch
 *                             chain can start on the other half.
 *   QGEMV_OPT_KSPLIT          0 (default): when K > 4096 and N * ceil(K / 2048) <= 4 Mi, each
 *                             CTA of the streaming kernel takes one 2048-wide K-column of a
 *                             range of rows (so it reads only that part of x) and the column
 *                             sums of a row meet in the handle's workspace, where the last
 *                             CTA of the range adds them in column order.  1: each CTA covers
 *                             every K-column of its rows and adds them in shared memory.
 *   QGEMV_OPT_GRID_PER_SM     0 (default): as many streaming CTAs per SM as fit, except
 *                             that with QGEMV_OPT_PDL a launch that covers K in one CTA and
 *                             has at most 16 rows per warp takes one CTA per SM; 1: one per
 *                             SM; 2: two per SM.  One per SM leaves the rest of each SM to
 *                             the next kernel of a programmatic-dependent-launch chain, whose
 *                             CTAs then fetch their first weights while this one finishes. */
typedef enum {
  QGEMV_OPT_FORCE_PATH = 0,
  QGEMV_OPT_RING_DEPTH = 2,
  QGEMV_OPT_ROWS_PER_STAGE = 3,
  QGEMV_OPT_SPIN_LIMIT_NS = 4,
  QGEMV_OPT_PDL = 5,
  QGEMV_OPT_TEST_STALL = 6,
  QGEMV_OPT_CTAS_PER_SM = 7,
  QGEMV_OPT_KSPLIT = 8,
  QGEMV_OPT_GRID_PER_SM = 9
} qgemv_option_t;

qgemv_status_t qgemv_set_option(qgemv_handle_t h, qgemv_option_t opt, int64_t value);

/* Describe the launch qgemv_run would make for (fmt, N, K) into `buf` (NUL-terminated,
 * at most `len` bytes): path, grid, block, warps per row, split, ring depth, shared
 * memory.  Returns the same validation status as qgemv_run without launching. */
qgemv_status_t qgemv_describe(qgemv_handle_t h, qgemv_format_t fmt, int64_t N, int64_t K, char* buf,
                              size_t len);

/* Compile-time build marker, checked by the Python binding at load (provenance). */
const char* qgemv_build_marker(void);

/* ---------------------------------------------------------------- layer entry points
 * The general form of the GEMV, y = alpha x.W^T + beta C (Q4_K page, section "What is a
 * GEMV", with C the output's previous contents), and launches over several matrices that
 * share one activation vector: the projections of a decoder layer that read the same x
 * (Q, K and V; the MLP's gate and up), which that page names as the GEMVs of each decoder
 * layer.  The MLP's gate/up pair can be combined as SwiGLU, h = silu(x.Wg^T) * (x.Wu^T)
 * with silu(g) = g / (1 + e^-g) (the gate of Llama/Qwen-style MLPs; the pages name the MLP
 * projections but not their activation). */

/* Output element types: fp32, or fp16 / bf16 rounded to nearest even from the fp32 result. */
typedef enum { QGEMV_OUT_F32 = 0, QGEMV_OUT_F16 = 1, QGEMV_OUT_BF16 = 2 } qgemv_out_t;

/* One matrix of qgemv_run_group.  For row n < N, with r the fp32 result of the row:
 *   swiglu = 0:  r = x . dequant(packed_W)[n, :]
 *   swiglu = 1:  r = silu(x . dequant(packed_W)[n, :]) * (x . dequant(packed_W_up)[n, :])
 *   y[n] = alpha * r + beta * y[n]    (y is not read when beta == 0; one rounding to `out`)
 * packed_W (and packed_W_up): device, qgemv_packed_bytes(fmt, N, K) bytes each, 16-byte
 * aligned; packed_W_up is ignored unless swiglu = 1.  y: device, N elements of type `out`,
 * 16-byte aligned, not overlapping x, any matrix or another problem's y. */
typedef struct {
  qgemv_format_t fmt;
  const void* packed_W;
  const void* packed_W_up;
  int64_t N;
  void* y;
  float alpha;
  float beta;
  qgemv_out_t out;
  int swiglu;
} qgemv_problem_t;

/* Maximum number of matrices in one qgemv_run_group call. */
#define QGEMV_MAX_GROUP 8

/* Runs `count` (1..QGEMV_MAX_GROUP) GEMVs that share x and K, as described by problems[]
 * (host array, read during the call only).  Formats may differ, except that x is bf16 when
 * the matrices are NVFP4 and fp16 otherwise, so NVFP4 cannot be mixed with the other
 * formats (QGEMV_ERR_INVALID_ARG).  K must be a multiple of every format's block length.
 * Matrices the streaming kernel takes (K a multiple of 256 and 16-byte rows) run in ONE
 * launch, each on a share of the CTAs in proportion to its bytes; the others get a
 * warp-per-row launch each.  Validation as qgemv_run for every matrix, all before any
 * launch; also INVALID_ARG for count out of range, a NULL problems, x or y, swiglu not 0/1,
 * swiglu = 1 without packed_W_up, or `out` out of range.  Asynchronous on `stream`, no
 * allocation; uses the handle's workspace like qgemv_run (one call at a time per handle).
 * Deterministic like qgemv_run. */
qgemv_status_t qgemv_run_group(qgemv_handle_t h, const void* x, int64_t K, int count,
                               const qgemv_problem_t* problems, cudaStream_t stream);

/* y = alpha * x . dequant(W)^T + beta * y for one matrix, y of type `out`: qgemv_run_group
 * with one problem (swiglu = 0).  alpha = 1, beta = 0, out = QGEMV_OUT_F32 computes what
 * qgemv_run does (through the grouped kernel, so the last bits may differ). */
qgemv_status_t qgemv_run_ex(qgemv_handle_t h, qgemv_format_t fmt, const void* x, const void* packed_W,
                            int64_t N, int64_t K, float alpha, float beta, void* y, qgemv_out_t out,
                            cudaStream_t stream);

/* ---------------------------------------------------------------- small batches
 * Y = X . dequant(W)^T for M = 1..QGEMV_MAX_BATCH activation vectors at once (the general
 * GEMV of the Q4_K page, "What is a GEMV", with x of shape (M, K) instead of (1, K)): every
 * packed weight is read and decoded once and serves all M vectors.  Every format uses the
 * tensor cores' mma.sync path (decoded weights go straight into the A fragments; the M vectors
 * fill the B operand) when M >= 4, or M >= 2 and N >= 4096 (below that two or three
 * single-vector launches are faster), with rows whose packed length is a multiple of 16 bytes
 * (K a multiple of 2048 for TQ1_0 and Q6_K, of 256 for the others) and M * N * ceil(K / 1024)
 * within the handle's workspace (4 Mi column sums); other calls run the single-vector path
 * once per vector.  Input domain of the tensor-core path: a Q8_0 weight d q is formed in
 * fp16, so weights must be below 65504 in magnitude (quantised model weights are many orders
 * of magnitude smaller); the single-vector path has no such limit. */
#define QGEMV_MAX_BATCH 8

/* x: device, M rows of K 16-bit values (fp16; bf16 for NVFP4), row-major, 16-byte aligned.
 * y: device, M rows of N fp32 values, row-major (y[m * N + n]), 16-byte aligned.
 * packed_W, N, K: as qgemv_run.  1 <= M <= QGEMV_MAX_BATCH, else QGEMV_ERR_INVALID_ARG.
 * Validation, asynchrony, workspace use and determinism as qgemv_run.  Each output obeys the
 * GEMV tolerance of its own vector. */
qgemv_status_t qgemv_run_batch(qgemv_handle_t h, qgemv_format_t fmt, const void* x, int M,
                               const void* packed_W, int64_t N, int64_t K, float* y,
                               cudaStream_t stream);

/* ---------------------------------------------------------------- many rows (prefill)
 * Y = X . dequant(W)^T for any number M >= 1 of activation rows: the matrix-matrix product
 * that the Mojo "fp4_gemv" page sets beside its GEMV (its opening description: a whole prompt
 * goes through the prefill path, a shared-memory tile feeding the matrix unit, while decode
 * at M = 1 is the GEMV).  NVFP4 with M > QGEMV_MAX_BATCH runs on the fifth-generation tensor
 * cores (tcgen05) when K is a multiple of 128 (of 64 when M > 128): tiles of 128 weight rows x
 * 64, 128 or 256 rows of X (by M), X brought in by TMA, the weights dequantised exactly to
 * bf16 into the MMA's A operand in tensor memory (e2m1 times an e4m3 scale has at most 6
 * significant bits), fp32 accumulation in tensor memory, K split over a thread-block cluster
 * when the tiles do not fill the GPU.  Every other call goes through qgemv_run_batch in
 * chunks of QGEMV_MAX_BATCH rows.
 *
 * x: device, M rows of K 16-bit values (fp16; bf16 for NVFP4), row-major, 16-byte aligned.
 * y: device, M rows of N fp32 values, row-major (y[m * N + n]), 16-byte aligned.
 * packed_W, N, K: as qgemv_run.  M < 1 gives QGEMV_ERR_INVALID_ARG; the tensor-core path
 * needs M, K < 2^31 (else QGEMV_ERR_BAD_SHAPE).  Asynchronous on `stream`, allocates
 * nothing; each output obeys the GEMV tolerance of its own row; repeated calls give identical
 * bits.  A wait in the tensor-core kernel that runs past QGEMV_OPT_SPIN_LIMIT_NS sets the
 * handle's error word (read by qgemv_check_error). */
qgemv_status_t qgemv_run_gemm(qgemv_handle_t h, qgemv_format_t fmt, const void* x, int64_t M,
                              const void* packed_W, int64_t N, int64_t K, float* y,
                              cudaStream_t stream);

/* ---------------------------------------------------------------- serving a batch of requests
 * What stands between the projections of a decode step that serves many requests: the pages of
 * a key-value cache are planned on the GPU (qgemv_page_plan), the QKV projection's rows are
 * rotated and written into them (qgemv_kv_store), each new token attends to its request's
 * pages (qgemv_attn_decode), and low-rank adapters are added to a projection's output
 * (qgemv_run_lora).  Every call is described by a struct (host memory, read during the call
 * only); nothing is allocated and nothing synchronises, so a step can be captured in a CUDA
 * graph.  Lengths, page tables, slots, positions and adapter numbers are read on the device;
 * one that is out of range is never used to address memory: what happens instead is said at
 * each entry point, and qgemv_check_error then reports QGEMV_ERR_BAD_INDEX.  Element types are
 * those of qgemv_out_t.  Strides are counted in elements.  The kernels are programmatic
 * dependent launches whatever QGEMV_OPT_PDL says: they may be set up while the kernel before
 * them on the stream ends, and read and write memory only after it.  Calls use the handle's
 * workspace like qgemv_run: one at a time per handle. */

/* A paged key-value cache.  k and v: device, page p at p * page_stride, inside it
 * [kv_heads][page_size][head_dim] elements, contiguous and 16-byte aligned (page_stride * element size a
 * multiple of 16 too; page_stride >= kv_heads * page_size * head_dim).  QGEMV_KV_E4M3: an e4m3
 * code c of token t and head h stands for c * scale[t, h]; k_scale and v_scale: device fp32,
 * [page][kv_heads][page_size], page p at p * scale_stride, 16-byte aligned with scale_stride a
 * multiple of 4 (ignored for the other types).
 * head_dim 64, 128 or 256; page_size 8 or a multiple of 16. */
typedef enum { QGEMV_KV_F16 = 1, QGEMV_KV_BF16 = 2, QGEMV_KV_E4M3 = 3 } qgemv_kv_t;
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride;
  int64_t scale_stride;
  int32_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  qgemv_kv_t type;
} qgemv_kv_cache_t;

/* Block tables and slot maps of one step.  Request r has cached[r] tokens in its pages and
 * brings fresh[r] new ones (both counted as 0 when negative); the new tokens of all requests
 * are numbered 0, 1, ... in request order.  Position i of request r lives in page
 * table[r][i / page_size]; a token that opens a page takes the next one from the top of the
 * stack free_pages[0 .. *free_count), in token order, and writes it into the table (other
 * entries of the table are left alone).  A token gets no slot when it lies past `capacity` or
 * past its row of the table, or when the stack is empty; neither do the later tokens of
 * that request.  A negative page in the table or the stack where a token's own page should be
 * is reported, and the token gets slot -1; it keeps its position, which later tokens of the
 * request follow, so lens and counts[1] count it.
 *   lens[r]       cached[r] + the new tokens of r that have a slot: the length to attend over
 *   offsets[r]    number of the first new token of request r; offsets[requests] = their total
 *                 (both at most 2^31 - 1, where larger ones stay)
 *   slots[t]      page * page_size + position % page_size, or -1    (t < capacity)
 *   positions[t]  position in the request, or -1
 *   owners[t]     request, or -1 past the total
 *   counts[0..3]  new tokens (at most 2^31 - 1), those with a slot, pages taken, pages that
 *                 were missing
 * free_pages and *free_count are only read: the caller lowers its count by counts[2].
 * positions, owners and offsets may be NULL.  All pointers device; slots, positions and
 * owners 16-byte aligned.  requests 0 .. 2^30, page_size >= 1, table_width >= 1 and <= table_stride,
 * 0 <= capacity < 2^31. */
typedef struct {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* table;
  int64_t table_stride;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* lens;
  int32_t* offsets;
  int64_t* slots;
  int32_t* positions;
  int32_t* owners;
  int32_t* counts;
  int64_t capacity;
  int32_t requests;
  int32_t table_width;
  int32_t page_size;
} qgemv_page_plan_t;

qgemv_status_t qgemv_page_plan(qgemv_handle_t h, const qgemv_page_plan_t* plan, cudaStream_t stream);

/* Rotates the q and k rows of `tokens` tokens and stores k and v in the cache.  Row t of q, k
 * and v starts at t * its stride and holds its heads one after another (the three can be
 * slices of one projection's output); element type `in`.
 *   rope          fp32 [rope_positions][rot_dim]: of each position rot_dim / 2 cosines, then
 *                 rot_dim / 2 sines; NULL: nothing is rotated.  Pair i (a, b) becomes
 *                 (a cos_i - b sin_i, b cos_i + a sin_i), with a, b the elements i and
 *                 i + rot_dim / 2 of a head, or 2 i and 2 i + 1 when interleaved = 1; elements
 *                 from rot_dim on are kept.  rot_dim: a multiple of 16, at most head_dim.
 *   positions[t]  -1: an unused row, whose q_out is zeros.  Another position outside the
 *                 rope table counts as -1 and is reported.
 *   slots[t]      as qgemv_page_plan gives them; -1: k and v of the row are not stored.
 *                 Another slot outside the cache counts as -1 and is reported.  No slot may
 *                 occur twice.
 *   q, q_out      may both be NULL; q_out [tokens][q_heads][head_dim] of type q_type (F16 or
 *                 BF16), row t at t * q_out_stride; it must not overlap q, k or v.
 * The rotation is computed in fp32 and rounded once to the cache's or q_out's type.  An E4M3
 * cache gets scale = max|x| / 448 of the token's head (1 where that is 0 or not finite, and at
 * least 2^-126) and the codes e4m3(x / scale), rounded to nearest even; infinities become +-448,
 * NaN stays NaN.
 * Pointers 16-byte aligned, row strides a multiple of 16 bytes.  slots, positions (and rope)
 * are needed also where no row is rotated. */
typedef struct {
  qgemv_kv_cache_t cache;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  void* q_out;
  int64_t q_out_stride;
  const int64_t* slots;
  const int32_t* positions;
  const float* rope;
  int64_t tokens;
  int32_t rope_positions;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t q_heads;
  qgemv_out_t in;
  qgemv_out_t q_type;
} qgemv_kv_store_t;

qgemv_status_t qgemv_kv_store(qgemv_handle_t h, const qgemv_kv_store_t* store, cudaStream_t stream);

/* Attention of one new token per request over its pages:
 *   out[r, g] = sum_t softmax_t(scale * q[r, g] . k[t]) v[t],   lo <= t < lens[r],
 *   lse[r, g] = log sum_t exp(scale * q[r, g] . k[t])           (natural logarithm)
 * with lo = max(0, lens[r] - window) (0 when window = 0), and k, v of kv head
 * g / (q_heads / kv_heads).  lens[r] counts the new token, whose k and v are stored.  A row
 * that sees no token, or whose every score is -inf, gives out = 0 and lse = -inf.
 *   q, out        [requests][q_heads][head_dim], row r at r * stride, `type` F16 or BF16 (that of
 *                 the cache, unless it is E4M3).
 *   table         [requests] rows of table_width pages at r * table_stride.  A page outside
 *                 the cache is skipped with its tokens and reported; a length past the table's
 *                 row counts as its end and is reported.
 *   lse           fp32 [requests][q_heads], or NULL.
 * Scores, the softmax and the sums are held in fp32 (16-bit products are exact); the weights
 * enter the second product as two 16-bit parts: 16 bits of each with BF16, 22 with F16 and E4M3, where
 * steps end at 2^-38 of the largest weight.  What lies in the cache outside the tokens
 * that a row sees, NaN included, does not reach it; an infinite value that it sees makes
 * its element infinite or NaN (the two parts of a weight may differ in sign).  Deterministic: the same inputs give the
 * same bits.  Uses the handle's workspace like qgemv_run.  q_heads a multiple of kv_heads;
 * requests 0 .. 2^30; out must not overlap q. */
typedef struct {
  qgemv_kv_cache_t cache;
  const void* q;
  int64_t q_stride;
  void* out;
  int64_t out_stride;
  float* lse;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  float scale;
  int32_t window;
  int32_t requests;
  int32_t table_width;
  int32_t q_heads;
  qgemv_out_t type;
} qgemv_attn_decode_t;

qgemv_status_t qgemv_attn_decode(qgemv_handle_t h, const qgemv_attn_decode_t* attn, cudaStream_t stream);

/* Low-rank adapters of many requests beside a shared projection: for row m with adapter
 * a = ids[m] of rank r = ranks[a],
 *   y[m, n] = base[m, n] + scales[a] * sum_{j < r} B[a, n, j] * (sum_k A[a, j, k] * x[m, k])
 * and y[m, n] = base[m, n] when ids[m] is -1 (or another number outside 0 .. adapters - 1,
 * which is reported).  base = NULL counts as zeros; base = y (same stride) adds in place.
 *   x             [rows][K], row m at m * x_stride; A [adapters][rank][K]; B [adapters][N][rank];
 *                 all of `type` F16 or BF16.
 *   ranks         [adapters], 0 .. rank (others are clamped); NULL: `rank` for all.  What lies
 *                 in A and B past an adapter's rank does not reach the result.
 *   scales        [adapters] fp32; NULL: 1.
 *   base, y       [rows][N] of type `out`, row m at m * y_stride (both).
 * Products are exact, sums in fp32; the inner sums enter the second product as two or three 16-bit
 * parts, with at least 21 bits of each whatever the size of the row's others; y is rounded once.  Infinities and NaN in an adapter or
 * a row of x make the results that use them infinite or NaN, and no others.  Deterministic.  rank a multiple
 * of 8, 8 .. 128; K a multiple of 8; x, A, B, base and y 16-byte aligned, x_stride a multiple
 * of 8. */
typedef struct {
  const void* x;
  int64_t x_stride;
  const void* A;
  const void* B;
  const int32_t* ids;
  const int32_t* ranks;
  const float* scales;
  const void* base;
  void* y;
  int64_t y_stride;
  int64_t rows;
  int64_t N;
  int64_t K;
  int32_t adapters;
  int32_t rank;
  qgemv_out_t type;
  qgemv_out_t out;
} qgemv_lora_t;

qgemv_status_t qgemv_run_lora(qgemv_handle_t h, const qgemv_lora_t* lora, cudaStream_t stream);

/* Capacity of qgemv_run_noalloc's scratch, in fp32 column sums: N * ceil(K / 2048) of them. */
#define QGEMV_NOALLOC_MAX_COLUMN_SUMS 262144

/* qgemv_run without a handle and without allocating anything.  (This entry point is part
 * of the library's interface only; the pages that describe the method have no
 * counterpart.)  It exists for callers that may not call cudaMalloc: code that runs under
 * a host application owning all device memory (a plug-in given fixed buffers), processes
 * whose allocator is capped or instrumented so a new allocation would fail or be refused,
 * and latency-critical paths where an allocation's implicit synchronisation is not
 * acceptable.  Those callers cannot use qgemv_create, which allocates the handle's
 * workspace.
 *
 * Computes y = x . dequant(W)^T exactly like qgemv_run with the split-K streaming kernel:
 * every CTA takes one 2048-wide K-column of a range of rows, and the column sums of a row
 * are added in column order.  Arguments, layouts and results are those of qgemv_run;
 * results are bitwise reproducible from call to call.  Shapes: K a multiple of 256 and at
 * most 32768, with packed rows a multiple of 16 bytes (K a multiple of 2048 for Q6_K and
 * TQ1_0), else QGEMV_ERR_BAD_SHAPE.  When K > 2048, N * ceil(K / 2048) must not exceed
 * QGEMV_NOALLOC_MAX_COLUMN_SUMS, else QGEMV_ERR_TOO_LARGE and nothing is launched.
 *
 * Scratch: fixed arrays in the library's device memory (1 MiB of column sums, 4 KiB of
 * counters), which every GPU that loads the library holds until the process exits.  All
 * calls on a device share them and they keep what the last call left: each call first
 * clears the counters with cudaMemsetAsync on `stream`, then launches.  Calls that may run
 * at the same time on the GPU (different streams, or host threads that do not order their
 * streams) race on the scratch and give wrong results; order them on one stream.
 *
 * The first call on a device (the current device) sets that device up: it looks up the
 * scratch arrays' device addresses with cudaGetSymbolAddress and sets the kernels'
 * shared-memory attribute.  Make that first call before any stream capture begins.
 * Asynchronous on `stream`; does not synchronise. */
qgemv_status_t qgemv_run_noalloc(qgemv_format_t fmt, const void* x, const void* packed_W, int64_t N, int64_t K,
                                 float* y, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H_ */
