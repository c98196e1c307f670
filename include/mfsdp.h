/*
 * mfsdp.h -- C ABI of the owner-local optimizer step on MI355X (gfx950).
 *
 * Source of the operations: "MatrixFSDP: communication-free matrix optimizers
 * under ZeRO-3 parameter sharding" (arxivlens page, Abstract; gist.science
 * technical summaries, section "Methodologie", part 1 "owner-shaped
 * placement").  Under owner-shaped ZeRO-3 placement every 2D weight lives whole
 * on one data-parallel owner and every other rank holds an empty shard for it;
 * after the ordinary gradient reduction the owner holds the whole gradient, so
 * its Muon step -- momentum, Newton-Schulz orthogonalization of the whole
 * matrix, update -- involves no communication.  Tensors that are not 2D
 * matrices are gathered on tail owners and updated there with AdamW.  This
 * library is that step on one GPU:
 *
 *   mfsdp_muon_step   -- Muon on the owner's list of whole matrices,
 *   mfsdp_adamw_tail  -- AdamW on a packed fp32 tail buffer.
 *
 * Further down: the owner planner, packed tails, Shampoo-type statistics, the
 * operators that make the gradients of experts' matrices and of an embedding
 * table, and those around them: routing, the exchange of rows, layer norm and
 * products in 8-bit floats.
 *
 * Conventions shared by every entry point
 *   - Every pointer named "device" is a device (HBM) address on the current
 *     HIP device.  The caller owns every buffer; the library never allocates
 *     or frees device memory.  Host pointers are read only during the call.
 *   - Work is enqueued asynchronously on `stream`; no call waits for device
 *     work to finish.
 *   - All arguments are validated before anything is enqueued.  On any
 *     status other than MFSDP_OK nothing has been modified, except for
 *     MFSDP_ERR_HIP, which is returned when the HIP runtime fails after work
 *     was enqueued (the contents of the outputs are then undefined).
 *   - mfsdp_last_error() returns a thread-local description of the last
 *     failure on the calling thread.  No C++ exception crosses this ABI.
 *   - Non-finite inputs are not checked: they propagate to the outputs.
 */
#ifndef MFSDP_H_
#define MFSDP_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mfsdp_status {
  MFSDP_OK = 0,
  MFSDP_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, bad scalar    */
  MFSDP_ERR_UNSUPPORTED = 2,      /* dtype or size this build cannot run   */
  MFSDP_ERR_WORKSPACE = 3,        /* workspace too small or misaligned     */
  MFSDP_ERR_ALIAS = 4,            /* two buffers that must not overlap do  */
  MFSDP_ERR_HIP = 5               /* the HIP runtime reported an error     */
} mfsdp_status_t;

typedef enum mfsdp_dtype {
  MFSDP_DTYPE_F32 = 0,  /* W, G, M and the Newton-Schulz iterates in fp32    */
  MFSDP_DTYPE_BF16 = 1  /* W, G, M in bf16; NS iterates bf16, fp32 accumulate */
} mfsdp_dtype_t;

/* Additive guard of the Frobenius normalization X0 = U / (||U||_F + eps). */
#define MFSDP_NS_EPS 1e-7f

/* Byte alignment required of every device buffer and of the workspace. */
#define MFSDP_ALIGNMENT 16

/*
 * One whole matrix owned by this rank (arxivlens Abstract: the owner holds the
 * complete 2D weight; its gradient arrives whole after the backward
 * reduction).  Stored row-major as rows x cols (rows = out_features),
 * contiguous, in the call's dtype.
 *
 *   weight      device, rows*cols, updated in place:
 *                 W <- (1 - lr*weight_decay) * W - lr * scale * O
 *   grad        device, rows*cols, read only
 *   momentum    device, rows*cols, updated in place: M <- beta*M + G
 *   update_out  device fp32 rows*cols, or NULL.  When given it receives O, the
 *               orthogonalized update before lr and scale.
 *   scale       the per-matrix update scale s (> 0, finite).  The common
 *               convention is sqrt(max(1, rows/cols)); the pages fix none.
 */
typedef struct mfsdp_matrix {
  void* weight;
  const void* grad;
  void* momentum;
  float* update_out;
  int64_t rows;
  int64_t cols;
  float scale;
} mfsdp_matrix_t;

/*
 * Workspace bytes that mfsdp_muon_step needs for this list (host call, no
 * device access).  The workspace holds the Newton-Schulz iterates of every
 * matrix (two m_pad x n_pad buffers and two m_pad x m_pad buffers per matrix,
 * m = min(rows, cols), n = max(rows, cols), padded to the 256-wide tile), the
 * per-block partial sums of the Frobenius norm and the launch descriptors.
 * Only rows, cols are read from `mats`.  n_mats == 0 gives 0 bytes.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT (null out / mats with n_mats > 0,
 * non-positive dims), MFSDP_ERR_UNSUPPORTED (dtype, or a size beyond the
 * 32-bit element indexing of the kernels).
 */
mfsdp_status_t mfsdp_muon_workspace_size(const mfsdp_matrix_t* mats,
                                         int64_t n_mats, mfsdp_dtype_t dtype,
                                         size_t* out_bytes);

/*
 * Owner-local Muon step over `n_mats` whole matrices (host array `mats`).
 *
 * For each matrix, in fp32 arithmetic (arxivlens Abstract: Muon orthogonalizes
 * momentum-smoothed updates with Newton-Schulz on the whole matrix):
 *   M' = beta*M + G                                  (stored to momentum)
 *   U  = G + beta*M'   (nesterov != 0)   or   U = M'
 *   X0 = U / (||U||_F + MFSDP_NS_EPS), transposed to m x n when rows > cols
 *   ns_steps times:  A = X X^T;  B = b*A + c*A*A;  X = a*X + B*X
 *   O  = X (transposed back)
 *   W' = (1 - lr*weight_decay)*W - lr*scale*O        (stored to weight)
 * With dtype BF16, X, A and B are rounded to bf16 (round to nearest even)
 * between the products, which accumulate in fp32.  Matrices are independent:
 * results do not depend on their order in the list or on how the library
 * groups them.
 *
 * workspace        device, >= mfsdp_muon_workspace_size bytes, 256-byte
 *                  aligned; contents are scratch and are overwritten.
 * n_mats == 0      (a rank that owns no matrix) returns MFSDP_OK, no work.
 * Streams: when a list has few rounds of tiles, the Newton-Schulz iterations
 * run as up to four flop-balanced groups of matrices.  The first group runs on
 * `stream`; the others run on auxiliary streams that the library owns, one
 * set per (device, caller stream), created on first use at the default
 * priority and kept until the process ends.  The auxiliary streams are forked
 * from `stream` with an event and joined back into it before the call
 * returns, so all the work is ordered after earlier work on `stream` and
 * before later work on it; calls on different caller streams share no
 * auxiliary stream.  The environment variable MFSDP_NS_GROUPS=1 keeps
 * everything on `stream`.  Calls may come from several host threads (one
 * caller stream per thread at a time); the pool lookup is guarded by a mutex.
 * Launch tables: each call uploads its descriptors and tile tables into the
 * workspace with hipMemcpyAsync from host memory that lives only during the
 * call (the HIP runtime stages such a copy before it returns).  A stream that
 * is being captured into a graph is therefore refused with
 * MFSDP_ERR_UNSUPPORTED, before anything is enqueued.
 * MFSDP_LOG=1 prints each call's launch plan (groups, tiles per launch,
 * padded shapes, workspace bytes) to stderr.
 * Validation: non-null weight/grad/momentum, rows, cols >= 1, 16-byte
 * aligned buffers, pairwise non-overlapping weight/grad/momentum/update_out/
 * workspace across the whole list, ns_steps in [0, 100], finite lr, beta,
 * weight_decay, a, b, c and scale, scale > 0.
 */
mfsdp_status_t mfsdp_muon_step(const mfsdp_matrix_t* mats, int64_t n_mats,
                               mfsdp_dtype_t dtype, float lr, float beta,
                               int nesterov, float weight_decay, int ns_steps,
                               float a, float b, float c, void* workspace,
                               size_t workspace_bytes, hipStream_t stream);

/*
 * The same step for callers that cannot allocate device memory: code that
 * may not call hipMalloc (tight serving loops, harnesses that forbid it, a
 * caller with no free HBM left to hand out a workspace).  It takes the
 * arguments of mfsdp_muon_step except the workspace, and uses instead a
 * static device array of MFSDP_NOALLOC_SCRATCH_BYTES (256 MiB) that the
 * library holds on every GPU it runs on, from the loading of its code object
 * on that GPU until the process ends.
 *   - A list whose workspace (mfsdp_muon_workspace_size) exceeds
 *     MFSDP_NOALLOC_SCRATCH_BYTES is refused with MFSDP_ERR_WORKSPACE before
 *     the device is touched: split the list, or use mfsdp_muon_step.
 *   - The call allocates no device or pinned host memory and creates no
 *     stream or event: every Newton-Schulz group runs on `stream` (results
 *     are bitwise those of mfsdp_muon_step, which does not depend on the
 *     grouping).  The only allocations are the host-side launch tables.
 *   - All calls on one GPU share that GPU's array, which keeps the last
 *     call's contents (nothing in it needs to start at zero: each call writes
 *     what it reads).  Calls that overlap on one GPU -- on two streams, or
 *     from two threads -- race on it and give undefined results; order them
 *     on one stream.
 *   - Like mfsdp_muon_step, a stream under graph capture is refused.
 * Validation and every other error are those of mfsdp_muon_step.
 */
#define MFSDP_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)

mfsdp_status_t mfsdp_muon_step_noalloc(const mfsdp_matrix_t* mats, int64_t n_mats,
                                       mfsdp_dtype_t dtype, float lr, float beta,
                                       int nesterov, float weight_decay, int ns_steps,
                                       float a, float b, float c, hipStream_t stream);

/*
 * Decoupled AdamW on a packed fp32 tail of n elements (arxivlens Abstract:
 * the tensors that are not 2D matrices go to tail owners in packed form and
 * keep the AdamW optimizer).
 * Elementwise, with t = step (>= 1):
 *   p  <- p * (1 - lr*weight_decay)
 *   m  <- beta1*m + (1-beta1)*g
 *   v  <- beta2*v + (1-beta2)*g*g
 *   p  <- p - lr * (m / (1-beta1^t)) / (sqrt(v / (1-beta2^t)) + eps)
 * param, exp_avg, exp_avg_sq are device fp32[n] updated in place, grad is
 * device fp32[n] read only; all 16-byte aligned and non-overlapping.
 * n == 0 (an owner with no tail) returns MFSDP_OK without touching the device.
 * Validation: non-null pointers for n > 0, n >= 0, step >= 1, finite
 * hyperparameters, beta1 and beta2 in [0, 1), eps >= 0; n > 2^40 returns
 * MFSDP_ERR_UNSUPPORTED.
 */
mfsdp_status_t mfsdp_adamw_tail(float* param, const float* grad,
                                float* exp_avg, float* exp_avg_sq, int64_t n,
                                float lr, float beta1, float beta2, float eps,
                                float weight_decay, int64_t step,
                                hipStream_t stream);

/*
 * Balance-aware owner planner (host only; touches no device).
 *
 * Source: arxivlens page, Methodology (a balance-aware owner planner assigns
 * ownership by bytes and by work); gist.science summaries, "Méthodologie",
 * part 2, first mechanism (a global planner chooses owners so that resident
 * bytes and optimizer work are balanced across the ranks).  The pages give no
 * algorithm; this one is greedy longest-processing-time-first scheduling
 * (Graham 1969) under a per-owner byte cap.
 *
 * Items are whole: a 2D matrix or a tail tensor, each going to exactly one of
 * n_ranks owners.
 *   cost_ms[n_items]   host, predicted optimizer-step time of each item on its
 *                      owner (for example measured per shape); finite, >= 0
 *   bytes[n_items]     host, resident bytes of each item on its owner (weight,
 *                      gradient and optimizer state); >= 0
 *   byte_slack         each owner's bytes stay within
 *                      cap = ceil((1 + byte_slack) * max(total/n_ranks, largest))
 *                      when any owner can take the item under it
 * In order of decreasing cost (ties: more bytes first, then lower index), each
 * item goes to the owner with the least predicted time among those it keeps
 * under the cap (ties: lower rank); when none can, to the owner with the
 * fewest bytes.  Without a binding cap the largest predicted time is within
 * (4/3 - 1/(3 n_ranks)) of the optimum.  Deterministic.
 * Outputs (host): owner[n_items] in [0, n_ranks); rank_ms[n_ranks] = summed
 * cost per owner; rank_bytes[n_ranks] = summed bytes per owner.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT (n_items < 0, n_ranks < 1, null
 * pointers, negative or non-finite cost, negative bytes or slack).
 */
mfsdp_status_t mfsdp_plan_owners(const double* cost_ms, const int64_t* bytes,
                                 int64_t n_items, int32_t n_ranks,
                                 double byte_slack, int32_t* owner,
                                 double* rank_ms, int64_t* rank_bytes);

/*
 * Packed tail layout (host only).  Source: arxivlens Abstract and gist.science
 * "Méthodologie", part 1: vectors and other non-2D tensors go, grouped, to a
 * tail owner, which runs AdamW on the packed buffer.
 * Tensor i of numel[i] fp32 elements occupies elements
 * [offsets[i], offsets[i] + numel[i]) of the packed buffer; segments follow
 * in order, each starting on a 16-byte (4-element) boundary.  *total is the
 * packed length (the last segment rounded up to 4).
 * Errors: MFSDP_ERR_INVALID_ARGUMENT (n < 0, null pointers, numel < 0).
 */
mfsdp_status_t mfsdp_tail_layout(const int64_t* numel, int64_t n,
                                 int64_t* offsets, int64_t* total);

/*
 * Gather tensors into a packed fp32 tail (device copy on `stream`).
 *   src[n]      host array of device pointers, tensor i of numel[i] fp32
 *               elements (4-byte aligned; may be NULL when numel[i] == 0)
 *   offsets[n]  host, element offsets in the packed buffer: multiples of 4,
 *               segments [offset, offset + round_up(numel, 4)) in bounds and
 *               pairwise disjoint (mfsdp_tail_layout gives such offsets)
 *   packed      device, packed_numel fp32 elements, 16-byte aligned; must not
 *               overlap any source
 * Each segment receives its tensor followed by zeros up to the next 4-element
 * boundary; elements outside every segment are left unchanged.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT, MFSDP_ERR_ALIAS (overlapping segments,
 * or a source overlapping the packed buffer), MFSDP_ERR_HIP.
 */
mfsdp_status_t mfsdp_tail_pack(const float* const* src, const int64_t* numel,
                               const int64_t* offsets, int64_t n, float* packed,
                               int64_t packed_numel, hipStream_t stream);

/*
 * Scatter a packed fp32 tail back into its tensors (device copy on `stream`):
 * dst[i][0 .. numel[i]) = packed[offsets[i] ..].  Same argument rules as
 * mfsdp_tail_pack; the destinations must not overlap each other or the
 * packed buffer (MFSDP_ERR_ALIAS).
 */
mfsdp_status_t mfsdp_tail_unpack(const float* packed, int64_t packed_numel,
                                 float* const* dst, const int64_t* numel,
                                 const int64_t* offsets, int64_t n,
                                 hipStream_t stream);

/*
 * Preconditioner statistics of Shampoo-type matrix optimizers on the owner.
 *
 * Source: gist.science summaries (French and Portuguese pages),
 * "Problématique" (Shampoo and SOAP, like Muon, take the whole 2D gradient
 * as input) and "Contributions clés", item "Généralité" (the owner-shaped
 * layout is not tied to one optimizer).  The arxivlens page names only Muon.  The pages give no formulas; the
 * statistics are the textbook Shampoo ones (Gupta, Koren and Singer 2018),
 * with SOAP's exponential moving average as the beta/alpha form.
 *
 * One whole gradient of the list, row-major rows x cols in the call's dtype:
 *   grad    device, read only
 *   left    device fp32 rows x rows, updated in place:  L <- beta*L + alpha*G G^T
 *   right   device fp32 cols x cols or NULL, updated:   R <- beta*R + alpha*G^T G
 * The products accumulate in fp32 from the stored gradient values (bf16 or
 * fp32); L and R stay exactly symmetric (the upper triangle is computed and
 * mirrored).  beta == 0 overwrites L and R without reading them.
 */
typedef struct mfsdp_stats_matrix {
  const void* grad;
  float* left;
  float* right;
  int64_t rows;
  int64_t cols;
} mfsdp_stats_matrix_t;

/* Workspace bytes for mfsdp_shampoo_stats (host only): two zero-padded copies
 * of each gradient (G and its transpose, 256-padded) and launch tables.
 * n_mats == 0 gives 0.  Errors: MFSDP_ERR_INVALID_ARGUMENT, MFSDP_ERR_UNSUPPORTED
 * (dtype, or a size beyond the 32-bit offsets of the kernels). */
mfsdp_status_t mfsdp_stats_workspace_size(const mfsdp_stats_matrix_t* mats,
                                          int64_t n_mats, mfsdp_dtype_t dtype,
                                          size_t* out_bytes);

/* Statistics update over the list, enqueued on `stream`.  workspace: device,
 * >= mfsdp_stats_workspace_size bytes, 256-byte aligned, scratch.  Like
 * mfsdp_muon_step, the call uploads its launch tables from host memory and
 * refuses a stream under graph capture (MFSDP_ERR_UNSUPPORTED).
 * Validation before any launch: rows, cols >= 1; non-null grad and left;
 * naturally aligned buffers; grad/left/right/workspace pairwise disjoint
 * across the list (MFSDP_ERR_ALIAS); finite beta and alpha. */
mfsdp_status_t mfsdp_shampoo_stats(const mfsdp_stats_matrix_t* mats, int64_t n_mats,
                                   mfsdp_dtype_t dtype, float beta, float alpha,
                                   void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/*
 * The gradients that the step takes.  Two kinds of tensors of a model have
 * gradients that are not one plain matrix product: the matrices of a mixture of
 * experts (a list of small whole matrices, each with the rows that were routed
 * to it), and the embedding table (a tail tensor under Muon's convention, in
 * the packed fp32 buffer of mfsdp_adamw_tail).  The calls below make them, with
 * the forward products they belong to and 8-bit copies of the activations that
 * the backward pass needs.
 *   - All of them are asynchronous on `stream`, allocate nothing, read offsets
 *     and tokens on the device, and can be captured into a graph (a graph
 *     keeps the workspace it was captured with: two graphs that may run at the
 *     same time need one each).
 *   - The calls that take a workspace share it in stream order: one host
 *     thread at a time per stream and workspace.
 *   - Results do not depend on timing: no atomics on sums.
 *   - Sums are fp32 throughout and rounded once, to the output's type.
 *   - Outputs must not overlap inputs, the workspace or each other
 *     (MFSDP_ERR_ALIAS); inputs may overlap inputs.
 *   - Buffers are aligned to their elements.  Rows that start on 16 bytes and
 *     widths of whole 16-byte groups take the fast kernels.
 *
 * Products grouped by expert.  Source: arxivlens Abstract (the owner holds
 * whole 2D weights and their whole gradients); gist.science "Contributions
 * cles" (matrix-wise optimizers on models with many small expert matrices).
 * The pages give no product: these are the linear layer and its derivatives.
 *   weight   device, n_experts x n x k, contiguous: W_e is the n x k row-major
 *            (out x in) matrix at weight + e*n*k, as mfsdp_muon_step takes it
 *   offsets  device int32, n_experts + 1, non-decreasing, in [0, rows]: rows
 *            offsets[e] <= r < offsets[e+1] of the activations go to expert e.
 *            An expert may have none.  Rows before offsets[0] and from
 *            offsets[n_experts] on belong to nobody: they are not read, and
 *            their output rows are left as they were.  Offsets are not checked
 *            on the host; the kernels clamp them to [0, rows] and take a
 *            decreasing pair as empty, so wrong ones give wrong results but no
 *            access outside the buffers.
 *   rows     rows of the activation buffers; ld_* row strides in elements
 * forward          y[r]  = x[r] W_e^T     (x: rows x k, y: rows x n)
 * input gradient   dx[r] = dy[r] W_e      (dy: rows x n, dx: rows x k)
 * weight gradient  dw_e  = beta*dw_e + sum_r dy[r]^T x[r], contiguous n_experts
 *                  x n x k in `dtype` or fp32 (dw_dtype).  beta == 0 does not
 *                  read dw; an expert without rows gets beta*dw_e.
 *                  Few or small matrices with many rows are summed in parts:
 *                  workspace (device, 256-byte aligned, scratch) then holds
 *                  mfsdp_grouped_linear_wgrad_workspace_size bytes; that may
 *                  be 0, and workspace NULL.
 * The checkpoint form takes x as codes and scales of mfsdp_ckpt_quantize
 * (contiguous, rows x k).  With dtype BF16 it multiplies them exactly; the
 * result is that of the weight gradient with the restored x.
 * n_experts == 0, and rows == 0 for the first two, return MFSDP_OK, no work.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT (negative counts, widths < 1, strides
 * smaller than rows, null or misaligned pointers, non-finite beta),
 * MFSDP_ERR_UNSUPPORTED (dtypes; n, k or strides above 2^22, rows above 2^30,
 * n_experts above 2^20, more than 2^23 tiles of the kernel that the call runs
 * -- see mfsdp_grouped_linear_tile; in the forward and input gradient through
 * registers, of 32 x 64 outputs), MFSDP_ERR_WORKSPACE,
 * MFSDP_ERR_ALIAS, MFSDP_ERR_HIP.
 */
mfsdp_status_t mfsdp_grouped_linear(const void* x, int64_t ld_x, const void* weight,
                                    const int32_t* offsets, int64_t n_experts, int64_t rows,
                                    int64_t n, int64_t k, mfsdp_dtype_t dtype, void* y,
                                    int64_t ld_y, hipStream_t stream);

mfsdp_status_t mfsdp_grouped_linear_dgrad(const void* dy, int64_t ld_dy, const void* weight,
                                          const int32_t* offsets, int64_t n_experts, int64_t rows,
                                          int64_t n, int64_t k, mfsdp_dtype_t dtype, void* dx,
                                          int64_t ld_dx, hipStream_t stream);

mfsdp_status_t mfsdp_grouped_linear_wgrad_workspace_size(int64_t n_experts, int64_t rows,
                                                         int64_t n, int64_t k,
                                                         mfsdp_dtype_t dtype, size_t* out_bytes);

mfsdp_status_t mfsdp_grouped_linear_wgrad(const void* dy, int64_t ld_dy, const void* x,
                                          int64_t ld_x, const int32_t* offsets, int64_t n_experts,
                                          int64_t rows, int64_t n, int64_t k, mfsdp_dtype_t dtype,
                                          void* dw, mfsdp_dtype_t dw_dtype, float beta,
                                          void* workspace, size_t workspace_bytes,
                                          hipStream_t stream);

mfsdp_status_t mfsdp_grouped_linear_wgrad_ckpt(const void* dy, int64_t ld_dy, const int8_t* codes,
                                               const uint8_t* scales, const int32_t* offsets,
                                               int64_t n_experts, int64_t rows, int64_t n,
                                               int64_t k, mfsdp_dtype_t dtype, void* dw,
                                               mfsdp_dtype_t dw_dtype, float beta,
                                               void* workspace, size_t workspace_bytes,
                                               hipStream_t stream);

/*
 * The kernel that a product of these sizes is computed with (host arithmetic,
 * no GPU): what a profile, or a test that means to run a certain kernel, checks
 * its sizes against.  rows_aligned: whether every operand row starts on 16
 * bytes.  A call that launches nothing gives zeros.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT, MFSDP_ERR_UNSUPPORTED, as the product's.
 */
typedef enum mfsdp_grouped_product {
  MFSDP_GROUPED_FORWARD = 0,
  MFSDP_GROUPED_DGRAD = 1,
  MFSDP_GROUPED_WGRAD = 2,
  MFSDP_GROUPED_WGRAD_CKPT = 3
} mfsdp_grouped_product_t;

typedef struct mfsdp_grouped_tile {
  int32_t rows, cols;     /* outputs of one workgroup                        */
  int32_t threads;        /* of one workgroup                                */
  int32_t wave_sets;      /* sets of waves that share each step of the sum   */
  int32_t lds_dma;        /* 1: operands go to LDS directly, 0: by registers */
  int32_t part_rows;      /* weight gradient in parts: rows of one, else 0   */
  int64_t workgroups;     /* of the launch, some of them without work        */
} mfsdp_grouped_tile_t;

mfsdp_status_t mfsdp_grouped_linear_tile(mfsdp_grouped_product_t product, int64_t n_experts,
                                         int64_t rows, int64_t n, int64_t k, mfsdp_dtype_t dtype,
                                         int rows_aligned, mfsdp_grouped_tile_t* out);

/*
 * Activation checkpoints in 8 bits: a copy of an activation, half (bf16) or a
 * quarter (fp32) of its size, kept from the forward to the backward pass.
 * Each row is cut into blocks of MFSDP_CKPT_BLOCK columns (the last may be
 * shorter); a block is held as whole numbers q in [-127, 127] and one power of
 * two 2^e, the smallest e >= -126 with max|x| <= 127 * 2^e, but 121 at most so
 * that q * 2^e stays finite:
 *   q = x / 2^e to the nearest, ties to even;   restored: q * 2^e
 * The error is at most 2^(e-1) (below 2^121 for |x| above 127.5 * 2^121, where
 * q stops at 127).  q * 2^e is exact in bf16 and fp32.
 *   x       device, rows x k, row stride ld_x, bf16 or fp32
 *   codes   device int8, rows x k, contiguous
 *   scales  device uint8, rows x ceil(k / MFSDP_CKPT_BLOCK): e + 127; 255 marks
 *           a block with an infinity or a NaN, which restores as NaN
 * rows == 0 returns MFSDP_OK, no work.  Errors as above.
 */
#define MFSDP_CKPT_BLOCK 128

mfsdp_status_t mfsdp_ckpt_quantize(const void* x, int64_t ld_x, int64_t rows, int64_t k,
                                   mfsdp_dtype_t dtype, int8_t* codes, uint8_t* scales,
                                   hipStream_t stream);

mfsdp_status_t mfsdp_ckpt_restore(const int8_t* codes, const uint8_t* scales, int64_t rows,
                                  int64_t k, mfsdp_dtype_t dtype, void* x, int64_t ld_x,
                                  hipStream_t stream);

/*
 * Embedding: out[i] = scale * table[token_i], in fp32 and rounded once.
 *   table   device, vocab x d, contiguous, bf16 or fp32 (a packed tail segment)
 *   tokens  device, n_tokens, int32 or int64 (token_bytes 4 or 8).  A token
 *           outside [0, vocab) stands for padding: its row is zero.
 *   out     device, n_tokens x d, row stride ld_out, bf16 or fp32
 * Its gradient, into the dense fp32 gradient of the table:
 *   grad[v] = beta*grad[v] + scale * sum_{i: token_i = v} dy[i]
 *   dy      device, n_tokens x d, row stride ld_dy, bf16 or fp32; the rows of
 *           padding tokens are not read
 *   grad    device fp32, vocab x d, contiguous.  beta == 0 does not read it
 *           (rows without a token become zero); beta == 1 leaves the rows
 *           without a token untouched.
 * Each row is summed over its tokens in the order of the list, in chunks of 64
 * of the sorted list when it has more than 64: the result depends on the
 * inputs alone.
 * workspace  device, >= mfsdp_embedding_grad_workspace_size bytes, 256-byte
 *            aligned, scratch; none is needed for n_tokens == 0.
 * Errors: as above, MFSDP_ERR_WORKSPACE, and MFSDP_ERR_UNSUPPORTED for vocab
 * above 2^31 - 1, n_tokens above 2^28, d or strides above 2^22, and for a
 * gradient of 2^24 or more chunks of 64 tokens and 2048 columns (512 where rows
 * are not whole 16-byte units).
 */
mfsdp_status_t mfsdp_embedding(const void* table, mfsdp_dtype_t table_dtype, int64_t vocab,
                               int64_t d, const void* tokens, int token_bytes, int64_t n_tokens,
                               float scale, void* out, int64_t ld_out, mfsdp_dtype_t out_dtype,
                               hipStream_t stream);

mfsdp_status_t mfsdp_embedding_grad_workspace_size(int64_t n_tokens, int64_t vocab, int64_t d,
                                                   size_t* out_bytes);

mfsdp_status_t mfsdp_embedding_grad(const void* dy, int64_t ld_dy, mfsdp_dtype_t dtype,
                                    const void* tokens, int token_bytes, int64_t n_tokens,
                                    int64_t vocab, int64_t d, float scale, float beta, float* grad,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Around the experts' products: which rows go where, the norms before them, and
 * the products in 8-bit floats.  The pages name experts and norm gains (tail
 * tensors of AdamW) but give no formulas: these are the usual ones.  The rules
 * of the gradient operators above hold here too (asynchronous, no allocation,
 * capturable, no atomics on sums, fp32 sums rounded once, outputs disjoint from
 * inputs, buffers aligned to their elements).  Rows may have any stride and
 * start at any element.
 *
 * Routing: the k experts of each token and their weights, from a row of logits x.
 *   s       softmax(x) or sigmoid(x)
 *   key     s + bias (no bias: s)
 *   groups  n_experts / groups neighbouring experts each; those with the
 *           top_groups largest sums of their two largest keys stay (groups == 1:
 *           all do)
 *   experts the k largest keys among those that stay, in descending order
 *   weights scale * s_j / (sum of the k chosen s + 1e-20), or scale * s_j without
 *           renormalize: the bias chooses and does not weigh
 * The choice is that of exact arithmetic on the logits and biases as stored, as
 * far as 64 bits tell it; ties go to the lowest index.  A NaN key is behind
 * -infinity; a row with a NaN or +infinity (softmax: or of -infinity alone) has NaN
 * weights where its scores are NaN, its experts are still k different ones.  Weights
 * are rounded in fp32 by the score, its share and the factor in turn: one expert
 * alone, renormalised, has exactly `scale` where its score is 2^-41 or more.
 *   logits   device, tokens x n_experts, row stride ld_logits, bf16 or fp32
 *   bias     device fp32, n_experts, or NULL
 *   mask     device, tokens bytes, or NULL: a token with 0 is padding, has experts
 *            -1 and weights 0, and its logits are not read
 *   experts  device int32, tokens x k;  weights device fp32, tokens x k
 * Gradient: of the logits, from that of the weights.  experts as chosen (an index
 * outside [0, n_experts) is none; one that is named twice counts twice); a token
 * without any has a row of zeros.  The choice itself has no gradient, and the
 * bias none.
 *   dweights device fp32, tokens x k;  dlogits device, as logits
 * tokens == 0 returns MFSDP_OK, no work.
 * Errors: MFSDP_ERR_INVALID_ARGUMENT (k outside [1, n_experts], groups that do
 * not divide n_experts, top_groups outside [1, groups] or with fewer than k
 * experts, strides smaller than rows, null or misaligned pointers, non-finite
 * scale), MFSDP_ERR_UNSUPPORTED (n_experts above 1024, k above 32, groups above
 * 64, 2^25 tokens or more, more than 2^30 choices), MFSDP_ERR_ALIAS,
 * MFSDP_ERR_HIP.
 */
typedef enum mfsdp_route_score {
  MFSDP_ROUTE_SOFTMAX = 0,
  MFSDP_ROUTE_SIGMOID = 1
} mfsdp_route_score_t;

mfsdp_status_t mfsdp_route(const void* logits, int64_t ld_logits, const float* bias,
                           const uint8_t* mask, int64_t tokens, int64_t n_experts, int64_t k,
                           mfsdp_dtype_t dtype, mfsdp_route_score_t scores, int64_t groups,
                           int64_t top_groups, int renormalize, float scale, int32_t* experts,
                           float* weights, hipStream_t stream);

mfsdp_status_t mfsdp_route_grad(const float* dweights, const void* logits, int64_t ld_logits,
                                const int32_t* experts, int64_t tokens, int64_t n_experts,
                                int64_t k, mfsdp_dtype_t dtype, mfsdp_route_score_t scores,
                                int renormalize, float scale, void* dlogits, int64_t ld_dlogits,
                                hipStream_t stream);

/*
 * Plan of a routing: the rows of the choices, sorted by expert, tokens in order
 * within one.
 *   experts  device int32, tokens x k; outside [0, n_experts): no row
 *   offsets  device int32, n_experts + 1: as the products grouped by expert take
 *            them; offsets[n_experts] is the number of rows in use
 *   place    device int32, tokens x k: the row of each choice, or -1
 * workspace  device, >= mfsdp_route_plan_workspace_size bytes (that may be 0, and
 *            workspace NULL), 256-byte aligned, scratch.
 * tokens == 0 gives offsets of zeros.  Errors as above, MFSDP_ERR_WORKSPACE; up to
 * 2^30 choices.
 */
mfsdp_status_t mfsdp_route_plan_workspace_size(int64_t tokens, int64_t k, int64_t n_experts,
                                               size_t* out_bytes);

mfsdp_status_t mfsdp_route_plan(const int32_t* experts, int64_t tokens, int64_t k,
                                int64_t n_experts, int32_t* offsets, int32_t* place,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Balance: bias[e] += rate where expert e has fewer choices than the mean, -= rate
 * where it has more (decided in whole numbers).
 *   bias    device fp32, n_experts, updated in place
 *   counts  device int32 or int64 (count_bytes 4 or 8), n_experts: choices of each
 *           expert, summed over the ranks where there are several
 */
mfsdp_status_t mfsdp_route_balance(float* bias, const void* counts, int count_bytes,
                                   int64_t n_experts, float rate, hipStream_t stream);

/*
 * Exchange of rows, by a plan's place (a row outside [0, rows) is none, and is
 * neither read nor written; rows of no choice are left as they were):
 *   dispatch          out[place[t][j]] = x[t]
 *   combine           y[t] = beta*y[t] + sum_j weights[t][j] * h[place[t][j]], j in order
 *                     (weights NULL: 1, which is dispatch's gradient); beta == 0
 *                     does not read y
 *   combine gradient  dh[place[t][j]] = weights[t][j] * dy[t]
 *                     dweights[t][j] = <dy[t], h[place[t][j]]>, 0 for none
 * x, y, dy: tokens x d; out, h, dh: rows x d, bf16 or fp32, any row stride.  Two
 * choices that name the same row are written in no order.
 * tokens == 0 returns MFSDP_OK, no work.  Errors as above; k up to 32, up to 2^30
 * choices and rows, d and strides up to 2^22.
 */
mfsdp_status_t mfsdp_route_dispatch(const void* x, int64_t ld_x, const int32_t* place,
                                    int64_t tokens, int64_t k, int64_t rows, int64_t d,
                                    mfsdp_dtype_t dtype, void* out, int64_t ld_out,
                                    hipStream_t stream);

mfsdp_status_t mfsdp_route_combine(const void* h, int64_t ld_h, const int32_t* place,
                                   const float* weights, int64_t tokens, int64_t k, int64_t rows,
                                   int64_t d, mfsdp_dtype_t dtype, float beta, void* y,
                                   int64_t ld_y, hipStream_t stream);

mfsdp_status_t mfsdp_route_combine_grad(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h,
                                        const int32_t* place, const float* weights, int64_t tokens,
                                        int64_t k, int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                                        void* dh, int64_t ld_dh, float* dweights,
                                        hipStream_t stream);

/*
 * Layer norm of rows of d values, in fp32 and rounded once:
 *   m = mean(x) (0 if not centered), v = mean((x - m)^2), xh = (x - m) / sqrt(v + eps)
 *   y = xh * weight + bias
 * (centered == 0 is the division by the root mean square, as in RMSNorm).
 *   x, y          device, rows x d, any row stride, bf16 or fp32
 *   weight, bias  device, d, bf16 or fp32 (weight_dtype; for example segments of a
 *                 packed tail); bias may be NULL
 * Gradients, with g = dy * weight; nothing of the forward is needed but x:
 *   dx      = (g - xh * mean(g * xh) - mean(g)) / sqrt(v + eps)   (the last mean if centered)
 *   dweight = beta*dweight + sum over rows of dy * xh     device fp32, d
 *   dbias   = beta*dbias + sum over rows of dy            device fp32, d, or NULL
 * for example segments of the packed gradient of mfsdp_adamw_tail; beta == 0 does
 * not read them.  Sums over rows are in a fixed order: equal inputs, sizes and
 * alignment give equal bits.
 * workspace  device, >= mfsdp_layer_norm_grad_workspace_size bytes, 256-byte
 *            aligned, scratch; none is needed for rows == 0.
 * rows == 0 returns MFSDP_OK; the gradients are then scaled by beta.
 * Errors as above; eps finite and >= 0; d and strides up to 2^22, rows up to 2^30.
 */
mfsdp_status_t mfsdp_layer_norm(const void* x, int64_t ld_x, const void* weight, const void* bias,
                                mfsdp_dtype_t weight_dtype, int64_t rows, int64_t d,
                                mfsdp_dtype_t dtype, int centered, float eps, void* y,
                                int64_t ld_y, hipStream_t stream);

mfsdp_status_t mfsdp_layer_norm_grad_workspace_size(int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                                                    int with_bias, size_t* out_bytes);

mfsdp_status_t mfsdp_layer_norm_grad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                     const void* weight, mfsdp_dtype_t weight_dtype, int64_t rows,
                                     int64_t d, mfsdp_dtype_t dtype, int centered, float eps,
                                     float beta, void* dx, int64_t ld_dx, float* dweight,
                                     float* dbias, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

/*
 * Products in 8-bit floats: e4m3 codes (OCP: 448 is the largest) with one power of
 * two 2^e per block of MFSDP_SCALED_BLOCK, the smallest e >= -126 with
 * max|v| <= 448 * 2^e, kept as the byte e + 127 (255: the block held an infinity or
 * a NaN, and its codes are NaN).  code = v / 2^e to the nearest, ties to even.  A
 * block is 128 columns of one row of activations, or 128 x 128 of a matrix.  Rows
 * of codes are filled up with zero codes to whole blocks: "filled" below is the
 * width rounded up to a multiple of 128.
 *   activations   x rows x k (any stride)     codes rows x filled k
 *                                             scales rows x ceil(k / 128)
 *   matrices      n_experts x n x k,          codes n_experts x n x filled k
 *                 contiguous                  scales n_experts x ceil(n/128) x ceil(k/128)
 *     transposed                              tcodes n_experts x k x filled n
 *                                             tscales n_experts x ceil(k/128) x ceil(n/128)
 *                 one call makes either copy or both (the same codes: either may
 *                 be NULL with its scales)
 *   product       y[r] = x[r] W_e^T for the rows offsets[e] <= r < offsets[e+1], the
 *                 values being code * 2^e; y rows x n, bf16.  The input gradient
 *                 is the same product, of dy's codes (depth n) with the transposed
 *                 ones (width k).  Sums: of eight neighbouring products 13 bits
 *                 below the largest are kept (the 8-bit MFMAs' own), those are
 *                 added in fp32, and the result is rounded once.
 * offsets, rows of nobody and limits are those of the products grouped by expert;
 * mfsdp_scaled_linear_tile names the kernel that sizes take, as
 * mfsdp_grouped_linear_tile does.  Codes are 16-byte aligned.  rows == 0 or n_experts == 0 returns MFSDP_OK, no
 * work.  Errors as above; widths up to 2^22 - 128.
 */
#define MFSDP_SCALED_BLOCK 128

mfsdp_status_t mfsdp_scaled_quantize(const void* x, int64_t ld_x, int64_t rows, int64_t k,
                                     mfsdp_dtype_t dtype, uint8_t* codes, uint8_t* scales,
                                     hipStream_t stream);

mfsdp_status_t mfsdp_scaled_quantize_weight(const void* weight, int64_t n_experts, int64_t n,
                                            int64_t k, mfsdp_dtype_t dtype, uint8_t* codes,
                                            uint8_t* scales, uint8_t* tcodes, uint8_t* tscales,
                                            hipStream_t stream);

mfsdp_status_t mfsdp_scaled_linear(const uint8_t* codes, const uint8_t* scales,
                                   const uint8_t* weight_codes, const uint8_t* weight_scales,
                                   const int32_t* offsets, int64_t n_experts, int64_t rows,
                                   int64_t n, int64_t k, void* y, int64_t ld_y,
                                   hipStream_t stream);

mfsdp_status_t mfsdp_scaled_linear_tile(int64_t n_experts, int64_t rows, int64_t n, int64_t k,
                                        mfsdp_grouped_tile_t* out);

/* Static, human-readable name of a status code. */
const char* mfsdp_status_string(mfsdp_status_t status);

/* Thread-local detail of the last failure on this thread ("" if none). */
const char* mfsdp_last_error(void);

/*
 * Kernel timing for measurement tools.  Kernels of the library fall into the
 * kinds below.  While timing is enabled on a thread, every launch that thread
 * makes is bracketed by a pair of hipEvents recorded on the launch stream
 * (not while that stream is being captured into a graph: its launches are
 * neither timed nor counted, then or when the graph is replayed);
 * mfsdp_timing_read synchronizes those events and returns, per kind, the
 * summed milliseconds and the number of launches since the last reset.
 * Events are created lazily by the library (no device-memory allocation) and
 * kept per thread.  Not needed for normal use.
 */
typedef enum mfsdp_kernel_kind {
  MFSDP_KERNEL_MOMENTUM = 0,  /* momentum + Nesterov + norm partials */
  MFSDP_KERNEL_NORM = 1,      /* per-matrix norm finalization        */
  MFSDP_KERNEL_GRAM = 2,      /* A = X X^T                           */
  MFSDP_KERNEL_POLY = 3,      /* B = b A + c A A                     */
  MFSDP_KERNEL_UPDATE = 4,    /* X = a X + B X, all but the last     */
  MFSDP_KERNEL_APPLY = 5,     /* apply when ns_steps == 0            */
  MFSDP_KERNEL_ADAMW = 6,     /* AdamW tail                          */
  MFSDP_KERNEL_FINAL = 7,     /* last update, applies W (2 launches) */
  MFSDP_KERNEL_STATS_PREP = 8,/* gradient copies for the statistics   */
  MFSDP_KERNEL_SYRK = 9,      /* L, R statistics products            */
  MFSDP_KERNEL_SMALL = 10,    /* whole NS chain + apply of small matrices */
  MFSDP_KERNEL_GROUPED = 11,  /* products grouped by expert          */
  MFSDP_KERNEL_CKPT = 12,     /* 8-bit checkpoints                   */
  MFSDP_KERNEL_EMBED = 13,    /* embedding lookup                    */
  MFSDP_KERNEL_EMBED_GRAD = 14, /* embedding gradient (all launches) */
  MFSDP_KERNEL_ROUTE = 15,      /* routing, its gradient, plan, balance */
  MFSDP_KERNEL_EXCHANGE = 16,   /* dispatch, combine and its gradient   */
  MFSDP_KERNEL_LAYER_NORM = 17, /* layer norm and its gradients         */
  MFSDP_KERNEL_SCALED = 18,     /* 8-bit floats and their products      */
  MFSDP_KERNEL_KINDS = 19
} mfsdp_kernel_kind_t;

mfsdp_status_t mfsdp_timing_enable(int enable);
mfsdp_status_t mfsdp_timing_reset(void);
mfsdp_status_t mfsdp_timing_read(mfsdp_kernel_kind_t kind, double* total_ms,
                                 int64_t* launches);

/*
 * Measurement only: the sustained bf16 MFMA rate of this GPU with no memory
 * traffic, the practical ceiling for the Newton-Schulz products (under
 * sustained MFMA load the clock settles below the one at which the dense peak
 * is quoted).  Launches `blocks` workgroups of 8 waves on `stream`; each wave
 * issues 8 * iters v_mfma_f32_32x32x16_bf16 (32768 flops each) on register
 * operands and writes one float to out[8 * block + wave] (device, blocks * 8
 * floats, 4-byte aligned).  The caller times the launch (for example with
 * hipEvents on `stream`).  Errors: MFSDP_ERR_INVALID_ARGUMENT (NULL or
 * misaligned out, blocks outside [1, 65536], iters outside [1, 2^20], or
 * blocks * iters above 2^28, which bounds a launch to about half a second),
 * MFSDP_ERR_HIP.
 */
mfsdp_status_t mfsdp_mfma_probe(float* out, int64_t blocks, int iters,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MFSDP_H_ */
