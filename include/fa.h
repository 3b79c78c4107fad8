/*
 * fa.h -- C ABI of the exact-attention library (libfa.so), sm_103a (GB300).
 *
 * The library computes exact scaled-dot-product attention, forward and
 * backward, tile by tile with an online softmax.  What it computes is the
 * plain definition: S = scale * Q K^T (optionally causal: key j <= query i),
 * P = softmax over each row of S, O = P V, LSE = ln sum_j exp(S_ij) -- the
 * two matrix products and softmax of "FlashAttention-4 : comment Together AI a
 * accéléré l'attention sur GPU Blackwell", section "Pourquoi l'approche
 * standard ne fonctionne plus"; the pages state that the tiled schedules leave
 * the mechanism unchanged ("FlashAttention-3 и FlashAttention-4", section
 * "Ключевая идея FlashAttention-3").  The backward pass is the chain rule of
 * the loss sum(O * dO): D = rowsum(dO * O), dP = dO V^T, dS = P * (dP - D),
 * dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO.
 *
 * Conventions shared by every entry point:
 *   - Tensors Q, K, V, O, dO, dQ, dK, dV are bf16, contiguous [B, H, N, d]
 *     (d fastest), device pointers, 16-byte aligned.  LSE is fp32 [B, H, N].
 *   - d must be 64 or 128.  Any N >= 0 is accepted; a ragged last tile is
 *     masked.  B, H, N of 0 are a no-op that returns FA_OK.
 *   - Queries and keys have the same length N, so "causal" is unambiguous.
 *   - The caller owns every input, output and workspace buffer; no entry
 *     point allocates or frees device memory.  The one piece of device
 *     memory the library holds is fa_bwd_noalloc's fixed scratch array,
 *     which lives in a module of its own and is loaded only by a process
 *     that calls fa_bwd_noalloc (see there).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *     default stream).  The return value reports argument validation and
 *     launch errors only.  A kernel that gives up on a bounded wait records
 *     FA_ERR_TIMEOUT in a device status word instead of hanging; read it
 *     with fa_last_device_status().  There is one status word per device,
 *     shared by every stream and host thread: after work on several
 *     streams, a timeout is reported to whichever caller reads it first.
 *   - Each kernel is launched so that it may start while the previous
 *     kernel in `stream` finishes (programmatic dependent launch); it waits
 *     for that work before touching any buffer.
 *   - Input and output buffers must not overlap.
 *   - Calls that may run at the same time (on several streams, or replayed by
 *     several graphs) need workspaces of their own.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null pointer, negative size, misaligned buffer   */
  FA_ERR_UNSUPPORTED = 2, /* a shape the kernels do not handle (d not 64/128)  */
  FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call or a launch failed      */
  FA_ERR_TIMEOUT = 4,     /* a kernel's bounded wait expired (device status)    */
  FA_ERR_WORKSPACE = 5,   /* the backward workspace is missing or too small     */
  FA_ERR_TOO_LARGE = 6    /* problem exceeds fa_bwd_noalloc's fixed scratch      */
} fa_status;

/*
 * Forward.  O = softmax(scale * Q K^T [masked]) V and, per row,
 * LSE = ln sum_j exp(scale * q_i . k_j) over the allowed keys (natural log of
 * the scaled scores).
 *   q, k, v : in,  bf16 [B, H, N, d]
 *   o       : out, bf16 [B, H, N, d]
 *   lse     : out, fp32 [B, H, N]
 *   scale   : the factor on Q K^T (usually 1/sqrt(d)); must be finite and > 0
 *   causal  : 0 = every key, 1 = key j <= query i
 *   workspace, workspace_bytes : optional device scratch owned by the caller
 *             (NULL / 0 = none).  With at least fa_fwd_workspace_bytes()
 *             bytes (256-byte aligned) the call may balance its last round
 *             of work (below); without it the result is the same, computed
 *             without that split.  Contents on entry do not matter.
 * Kernels: TMA-staged Q/K/V tiles, tcgen05 MMAs accumulating S and O in
 * tensor memory, warp-specialised load / MMA / softmax roles, polynomial exp2
 * on the FMA pipe selectable beside the MUFU unit (fa_set_exp2_poly_share),
 * O rescaled only when a row max grows past a threshold (FlashAttention-4
 * abstract, items 1-3).  One persistent CTA per SM walks the (batch, head,
 * 256-query block) work items.  Non-causal, when the last round of items
 * would leave SMs idle and a workspace is given, those items are cut into
 * key ranges merged by log-sum-exp (as fa_fwd_splitkv does), their fp32
 * partials kept in the workspace.
 * Returns FA_ERR_WORKSPACE for a non-NULL workspace that is short or not
 * 256-byte aligned.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
           int N, int d, float scale, int causal, void* workspace, size_t workspace_bytes,
           void* stream);

/*
 * Bytes of optional workspace fa_fwd uses to split its last partial round of
 * work items on the current device (the split depends on the device's SM
 * count): fp32 partial O and LSE of the split items.  0 when no split applies
 * (causal problems, problems whose items fill whole rounds, short key
 * ranges) or for empty or unsupported shapes.
 */
size_t fa_fwd_workspace_bytes(int B, int H, int N, int d, int causal);

/*
 * Share of the bf16 forward's exponentials evaluated in software on the FMA
 * pipe: per_octet of every 8 exponentials of a row tile (0..3) go to a
 * degree-3 polynomial exp2 (2^x = 2^round(x) * p(x - round(x)), max relative
 * error 1.01e-4), the rest to the MUFU ex2 unit ("Программная эмуляция
 * экспоненты" of "FlashAttention-3 и FlashAttention-4"; FlashAttention-4
 * abstract, item 2).  Process-wide, for calls made after it; the initial
 * value is 0, or FA_FWD_POLY_PER_OCTET from the environment.  On GB300 the
 * MUFU unit is not the forward's limit and every share above 0 measured
 * slower.  Returns FA_ERR_INVALID_ARG outside 0..3.
 * fa_get_exp2_poly_share() returns the current value.
 */
int fa_set_exp2_poly_share(int per_octet);
int fa_get_exp2_poly_share(void);

/*
 * 2-CTA forward: the same operation, arguments and errors as fa_fwd, computed
 * by pairs of CTAs (a cluster of two on one TPC) that share every product as
 * one M = 256 tcgen05 MMA (cta_group::2): each CTA keeps two of the pair's
 * four 128-row query tiles with their S, P and O in its own tensor memory,
 * and loads half of every K tile (64 keys) and half of every V tile (64 of
 * the d columns), so each K/V tile crosses from L2 into the SM pair once.
 * ("FlashAttention-3 и FlashAttention-4", section "Режим 2-CTA MMA": two
 * CTAs on one matrix operation halve the shared-memory load; FlashAttention-4
 * abstract, items 1 and 3: larger tiles, 2-CTA MMA.)  A work item is 512
 * query rows of one (batch, head); there is no key-range split.  Only
 * d = 128 (others return FA_ERR_UNSUPPORTED).  Results are bit-identical to
 * fa_fwd's.  On GB300 it runs slower than fa_fwd (shared memory is not what
 * limits the forward, and every product of the pair waits on operands and P
 * of both CTAs); it is kept as the measured variant.
 */
int fa_fwd_2cta(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int N, int d, float scale, int causal, void* stream);

/*
 * Split-KV forward: the same results as fa_fwd (within rounding), computed
 * with each query tile's key tiles cut into num_splits contiguous ranges
 * that run as separate work items, for problems with too few (batch, head,
 * query-block) items to fill the GPU, such as long context with few heads.
 * Each range leaves O normalised over the range and its LSE (fp32) in the
 * workspace; a merge kernel combines them by log-sum-exp:
 *   LSE = ln sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s
 * ("FlashAttention-4: Algorithm and Kernel Pipelining Co-Design", abstract:
 * long-context attention; the merge is the online-softmax rescaling of the
 * same pages applied across ranges).
 *   num_splits: 1 .. ceil(N / 128); 1 runs fa_fwd (workspace unused).
 *   workspace : at least fa_fwd_splitkv_workspace_bytes() bytes, 256-byte
 *               aligned, owned by the caller, contents on entry irrelevant.
 * Errors as fa_fwd, plus FA_ERR_INVALID_ARG for num_splits out of range and
 * FA_ERR_WORKSPACE for a missing, short or misaligned workspace.
 */
size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int N, int d, int num_splits);
int fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                   int N, int d, float scale, int causal, int num_splits, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * FP8 forward with incoherent processing ("FlashAttention-3 и
 * FlashAttention-4", section "Поддержка FP8 с контролем ошибок": a cheap
 * transform spreads outliers over the coordinates before quantisation).
 * Inputs and outputs as fa_fwd (bf16 Q, K, V; bf16 O; fp32 LSE), d = 128.
 * The call first rotates Q and K along the head dimension with the
 * orthogonal R = diag(sigma) H / sqrt(128) (H Sylvester-Hadamard, sigma a
 * fixed +-1 pattern) when rotate = 1, which leaves Q K^T unchanged, and
 * quantises to e4m3 in the workspace (Q one scale per row, K and V one per
 * (batch, head); V stored transposed); both products then run as e4m3
 * tensor-core MMAs with fp32 accumulation, P quantised to e4m3 as well.
 * The result approximates fa_fwd's to FP8 precision (about 5% relative
 * Frobenius error on O for N(0,1) inputs).
 *   rotate    : 1 = rotate Q and K (incoherent processing), 0 = plain FP8
 *   workspace : fa_fwd_fp8_workspace_bytes() bytes, 256-byte aligned: the
 *               e4m3 operands and their scales, then the partials of the
 *               last-round split fa_fwd makes on the current device
 * Returns FA_ERR_UNSUPPORTED for d != 128, FA_ERR_WORKSPACE for a missing,
 * short or misaligned workspace, FA_ERR_INVALID_ARG for rotate not 0 or 1.
 */
size_t fa_fwd_fp8_workspace_bytes(int B, int H, int N, int d);
int fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int N, int d, float scale, int causal, int rotate, void* workspace,
               size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace fa_bwd needs: fp32 D = rowsum(dO * O) [B, H, N]
 * and the fp32 dQ accumulator [B, H, N, d], each 256-byte aligned.
 * Returns 0 for empty or unsupported shapes.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward of the loss sum(O * dO).
 *   q, k, v   : in,  bf16 [B, H, N, d]  (the forward's inputs)
 *   o, lse    : in,  the forward's outputs (bf16 [B,H,N,d], fp32 [B,H,N])
 *   dout      : in,  bf16 [B, H, N, d]
 *   dq, dk, dv: out, bf16 [B, H, N, d]
 *   workspace : device scratch of at least fa_bwd_workspace_bytes(B,H,N,d)
 *               bytes, 256-byte aligned, owned by the caller; its contents on
 *               entry do not matter and are overwritten.
 * Three kernels run in stream order: D and dQ-accumulator zeroing; the
 * key/value-stationary main kernel (S and dP recomputed in tensor memory, dK
 * and dV accumulated there, dQ added with fp32 atomics -- the backward's
 * "reductions and atomic updates" of "FlashAttention-3 и FlashAttention-4",
 * section "Режим 2-CTA MMA"); and dQ conversion to bf16.
 * Returns FA_ERR_WORKSPACE when workspace is NULL or workspace_bytes is short.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
           const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
           float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

/*
 * 2-CTA backward: the same operation, arguments, workspace and errors as
 * fa_bwd, computed by pairs of CTAs (a cluster of two on one TPC) that own two
 * consecutive 128-key tiles of one head and share every product as one
 * tcgen05 cta_group::2 MMA ("FlashAttention-3 и FlashAttention-4", section
 * "Режим 2-CTA MMA": two CTAs on one matrix operation halve the
 * shared-memory operand traffic and the backward's atomic updates;
 * FlashAttention-4 abstract, item 3).  S^T, dP^T, dV and dK are M = 256
 * products in which each CTA loads half of every Q / dO operand;
 * dQ^T = K^T dS^T is one product over the pair's 256 keys, each CTA adding
 * its 64 rows of d, so dQ takes one fp32 addition per element per 256 keys
 * instead of per 128.  Each compute warpgroup writes its half of dS into the
 * shared memory of the CTA that needs it (distributed shared memory).
 * Only d = 128 (others return FA_ERR_UNSUPPORTED).  dK and dV equal fa_bwd's
 * within rounding; dQ within the order of its fp32 additions.
 */
int fa_bwd_2cta(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace fa_bwd_deterministic needs: fp32 D [B, H, N]
 * (256-byte aligned).  Returns 0 for empty or unsupported shapes.
 */
size_t fa_bwd_deterministic_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward with results that are bit-identical from run to run.  The pages
 * single out the backward's dQ reduction (fp32 atomic adds from every key
 * tile, whose order varies between runs) as a cost ("FlashAttention-3 и
 * FlashAttention-4", section "Режим 2-CTA MMA").  Here dK and dV come from
 * fa_bwd's key-stationary kernel without its dQ product, and dQ from a
 * second, query-stationary kernel that recomputes P and dS for its query
 * tile and adds dS K over the key tiles in order (causal: key tiles 0..i for
 * query tile i) in tensor memory.  dK and dV are deterministic in both entry
 * points (each key tile owns its rows and accumulates them in a fixed order)
 * and equal to fa_bwd's bit for bit.
 * Same arguments, results and errors as fa_bwd; the workspace must hold
 * fa_bwd_deterministic_workspace_bytes(B, H, N, d) bytes.  Slower than fa_bwd
 * by the recomputed S and dP products.
 */
int fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Backward without any allocation, for callers that cannot allocate device
 * memory: plugin hosts that hand a library its input and output buffers but
 * no allocator and no workspace, and latency-critical loops where a
 * cudaMalloc/cudaFree would synchronise the device.  The pages describe no
 * such entry point; it has no counterpart there.
 *
 * Same arguments and results as fa_bwd, minus the workspace: the scratch
 * (D and the fp32 dQ accumulator) lives in one fixed array of
 * FA_NOALLOC_SCRATCH_BYTES (96 MiB) of device memory inside the library.
 * The array sits in a module of its own, which the CUDA runtime loads on a
 * device at the process's first fa_bwd_noalloc call there (with the
 * runtime's default lazy module loading; CUDA_MODULE_LOADING=EAGER loads it
 * with the library); from then on that device keeps it until the process
 * exits.  Processes that never call fa_bwd_noalloc do not hold it.
 * Problems whose fa_bwd_workspace_bytes() exceeds it (at d = 128 roughly
 * B*H*N > 195,000 rows, at d = 64 > 380,000) return FA_ERR_TOO_LARGE.
 * The call allocates nothing: no cudaMalloc, cudaFree or allocating library
 * routine.  Its first call on a device looks up that device's address of the
 * array (with that device current); make that first call before any stream
 * capture.  The array keeps the last call's contents; the call itself
 * zeroes the part that must start at zero.  All calls share the one array,
 * so calls that overlap on the GPU (on different streams, or from several
 * threads) race and give wrong results: serialise them.
 */
#define FA_NOALLOC_SCRATCH_BYTES (96ull << 20)
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   float scale, int causal, void* stream);

/*
 * Causal attention with a sliding window, first tokens that stay visible, and
 * key/value heads shared by groups of query heads.  Query i sees the keys
 *   j <= i  with  i - j < window  or  j < sinks,
 * and query head h reads key head h / (H / Hkv).
 *   q, o   : bf16 [B, H, N, d]; k, v: bf16 [B, Hkv, N, d]; lse: fp32 [B, H, N]
 *   Hkv    : key/value heads; H is a multiple of it
 *   window : keys that a query sees, itself included, at least 1; from N on
 *            every key before it (plain causal attention, with shared heads)
 *   sinks  : first keys that every query sees besides, 0 .. 128 (more:
 *            FA_ERR_UNSUPPORTED)
 * Otherwise as fa_fwd with causal = 1.  Every element of K and V has to be
 * finite, also in padding rows of a batch: a masked pair's weight is an exact
 * 0, and 0 times an infinity or a NaN is not.
 */
int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                  int Hkv, int N, int d, float scale, int window, int sinks, void* stream);

/*
 * Backward of fa_fwd_window, as fa_bwd: dk and dv, bf16 [B, Hkv, N, d], are
 * summed over the query heads of the group (in fp32, in an order that does not
 * vary: bit-identical from run to run; dq within the order of its fp32
 * additions).
 *   workspace : fa_bwd_window_workspace_bytes() bytes for the current device,
 *               256-byte aligned: fa_bwd's, then, where queries see first tokens
 *               that their windows have left, the parts of those tokens' dK
 *               and dV, then the parts of key tiles whose query tiles are
 *               split over SMs that a last round of work would leave idle
 */
size_t fa_bwd_window_workspace_bytes(int B, int H, int Hkv, int N, int d, int window, int sinks);
int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dout, void* dq, void* dk, void* dv, int B, int H, int Hkv, int N, int d,
                  float scale, int window, int sinks, void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * Packed sequences: the rows of several sequences of different lengths, one after
 * another in one tensor, without padding between them.  Sequence b holds the rows
 * cu_seqlens[b] .. cu_seqlens[b+1]-1; rows before the first and from the last
 * one's end on are padding: they are not looked at, and outputs keep there what
 * they held.
 *
 * A row tensor has `heads` rows of d bf16 values per token, at
 * data + token * row + head * head (strides in elements, multiples of 8; data
 * 16-byte aligned), so rows that a fused projection leaves, or views of a fused
 * gradient, need no copy.  Rows of different tokens or heads do not overlap (no
 * stride of 0; strides of a single token or head do not matter).
 */
typedef struct {
  void* data;
  long long row;  /* from a token to the next */
  long long head; /* from a head to the next */
} fa_rows;

/*
 * A plan of packed sequences: the tiles of all sequences, those of most work
 * first, and each row's position in its sequence, in device memory that the
 * caller owns.  It is made from cu_seqlens by one kernel, once for a batch, and read
 * by every fa_fwd_packed and fa_bwd_packed on rows of this batch (any number of
 * heads, any layer).  cu_seqlens is not needed afterwards.
 *   cu_seqlens : in,  int [sequences + 1], read on the device: a captured graph
 *                serves whatever it holds at each replay
 *   rows       : rows of the tensors; 0 <= cu_seqlens[0] <= ... <=
 *                cu_seqlens[sequences] <= rows.  The kernel checks this: offsets
 *                that do not run forwards within the rows give a plan of no
 *                sequence, and FA_ERR_INVALID_ARG is recorded in the device
 *                status word.
 *   causal     : 1 = a row sees its sequence's rows up to itself, 0 = all of
 *                them, in every call with this plan
 *   plan       : out, fa_packed_plan_bytes() bytes, 256-byte aligned.  The rows'
 *                positions are at FA_PACKED_POSITIONS bytes into it: int [rows],
 *                -1 for padding (fa_rotate's `positions`).
 * At most 2^30 rows and 2^30 sequences (FA_ERR_UNSUPPORTED); empty sequences are
 * allowed.
 */
#define FA_PACKED_POSITIONS 256
size_t fa_packed_plan_bytes(int sequences, int rows);
int fa_packed_plan(const int* cu_seqlens, int sequences, int rows, int causal, void* plan,
                   size_t plan_bytes, void* stream);

/*
 * Attention within each of several packed sequences, key/value heads shared by groups of
 * query heads (query head h reads key head h / (H / Hkv)):
 *   O = softmax(scale q K^T) V over the rows that a row sees, LSE as fa_fwd.
 *   plan            : of these rows (fa_packed_plan); a kernel that meets another one
 *                     computes nothing and records FA_ERR_INVALID_ARG
 *   sequences, rows : as the plan was made with
 *   q, o            : in, out: row tensors of H heads; k, v: of Hkv heads, H a
 *                     multiple of Hkv
 *   lse             : out, fp32 [rows, H]
 *   d               : 64 or 128
 *   workspace       : optional (NULL, 0 = none): with fa_fwd_packed_workspace_bytes()
 *                     bytes on the current device, 256-byte aligned, contents on entry
 *                     irrelevant, a call with too few work items for the SMs (a
 *                     long prompt of few heads) cuts them into key ranges,
 *                     joined by a second kernel as fa_fwd_splitkv's.  0 bytes where
 *                     that does not apply.  Whether it does is decided by the mean
 *                     length, rows / sequences, empty sequences counted: a long
 *                     sequence beside many short or empty ones is not cut.
 *                     Calls in flight at once need one each.
 *                     FA_ERR_WORKSPACE for a short or misaligned one.
 * K and V have to be finite in the rows of a sequence that hold a row's later keys
 * (a masked pair's weight is an exact 0, and 0 times an infinity or a NaN is not);
 * what other sequences and padding rows hold does not matter.
 */
size_t fa_fwd_packed_workspace_bytes(int sequences, int rows, int H, int Hkv, int d);
int fa_fwd_packed(const void* plan, int sequences, int rows, const fa_rows* q, const fa_rows* k,
                  const fa_rows* v, const fa_rows* o, float* lse, int H, int Hkv, int d, float scale,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of fa_fwd_packed, as fa_bwd: gradients of sum(O * dO); dk and dv
 * are summed over the query heads of the group (in fp32, in an order that does not
 * vary: bit-identical from run to run; dq within the order of its fp32 additions).
 *   o, lse     : in,  the forward's outputs
 *   dout, dq   : in, out: row tensors of H heads; dk, dv: out, of Hkv heads
 *   workspace  : fa_bwd_packed_workspace_bytes() bytes, 256-byte aligned, contents
 *                on entry irrelevant: fp32 D and LSE by heads, the dQ
 *                accumulator and, where key tiles are split over SMs (by the
 *                current device's SM count and the mean length, empty
 *                sequences counted), the parts of dK and dV.  0 for
 *                empty or unsupported shapes.
 * What rows of the other sequences and padding rows hold does not matter; a
 * sequence's own rows have to be finite, all of them.  rows * H up to 2^31 - 1
 * (FA_ERR_UNSUPPORTED).
 */
size_t fa_bwd_packed_workspace_bytes(int sequences, int rows, int H, int Hkv, int d);
int fa_bwd_packed(const void* plan, int sequences, int rows, const fa_rows* q, const fa_rows* k,
                  const fa_rows* v, const fa_rows* o, const float* lse, const fa_rows* dout,
                  const fa_rows* dq, const fa_rows* dk, const fa_rows* dv, int H, int Hkv, int d,
                  float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotates Q and K rows by their positions (before fa_fwd_packed), or turns their
 * gradients back (after fa_bwd_packed).
 *   q, q_out  : in, out: row tensors of H heads, or both NULL (H = 0)
 *   k, k_out  : the same of Hkv heads
 *               An output may be its own input (the same data and strides), and may
 *               not overlap it otherwise.
 *   positions : in, int [rows]; a row of negative position is left as it was
 *   rope      : in, fp32 [rope_len, rot]: row p holds cos of the rot/2 angles of
 *               position p, then their sines (any pair of factors: a table for
 *               long contexts may be scaled).  A position past the table:
 *               the row is left as it was and FA_ERR_INVALID_ARG is recorded.
 *   rot       : elements of a row that are rotated, a multiple of 16 from 16 to d; the
 *               others are copied
 *   interleaved, and the arithmetic: as fa_paged_append
 *   backward  : 0 = rotate; 1 = the transpose, x_a = x'_a cos + x'_b sin, x_b =
 *               x'_b cos - x'_a sin: the gradient of x from that of x'
 */
int fa_rotate(const fa_rows* q, const fa_rows* q_out, int H, const fa_rows* k, const fa_rows* k_out,
              int Hkv, const int* positions, int rows, int d, const float* rope, int rope_len, int rot,
              int interleaved, int backward, void* stream);

/*
 * A paged key/value cache.  The cache is an array of num_pages * Hkv blocks;
 * block (page, head) holds page_size consecutive positions of one key head of
 * one sequence: their K rows, then their V rows.
 *   FA_CACHE_BF16: rows of d bf16 values.
 *   FA_CACHE_FP4 : the K rows' codes (d/2 bytes a row, e2m1, the even element
 *                  in the low four bits), the K rows' scales (d/16 bytes a
 *                  row, e4m3, one per 16 consecutive elements), then V's codes
 *                  and scales.  An element stands for code * scale * g, with
 *                  g the head's factor (k_scale, v_scale).
 * Position p of sequence b is in page page_table[b * max_pages + p / page_size],
 * row p % page_size.  New rows come as a ragged batch: the rows cu_new[b] ..
 * cu_new[b+1]-1 of the row tensors belong to sequence b and are its last ones,
 * at the positions seq_lens[b] - (cu_new[b+1] - cu_new[b]) .. seq_lens[b]-1,
 * so seq_lens counts the new rows.  Rows from cu_new[B] on are padding.
 *
 * page_table, seq_lens, cu_new, k_scale and v_scale are read on the device
 * (a captured graph serves whatever they hold at each replay) and so cannot be
 * checked by the call.  The kernels check them: a position past its sequence's
 * pages (or the rotation's table), a page outside the cache, all rows of a
 * sequence that reach past the tensors' rows, start before them or run backwards
 * are skipped, and FA_ERR_INVALID_ARG is recorded in the device status word.  Pages that one call writes must belong to one position
 * of one sequence each; pages that are only read may be shared.
 */
typedef enum {
  FA_CACHE_BF16 = 0,
  FA_CACHE_FP4 = 1
} fa_cache_format;

typedef struct {
  void* pages;            /* num_pages * Hkv blocks of fa_paged_block_bytes, 16-byte aligned */
  const int* page_table;  /* [B, max_pages] */
  const int* seq_lens;    /* [B] */
  const float* k_scale;   /* FA_CACHE_FP4: [Hkv], finite and > 0, or NULL = 1; else NULL */
  const float* v_scale;   /* the same for V */
  int format;             /* fa_cache_format */
  int B;                  /* sequences */
  int Hkv;                /* key/value heads */
  int d;                  /* 64 or 128 */
  int num_pages;
  int page_size;          /* 16, 32, 64 or 128 */
  int max_pages;          /* pages of a sequence at most */
} fa_paged_cache;

/* Bytes of one block: a page's K and V rows of one head.  0 for a format,
 * page size or head dim that the cache does not have. */
size_t fa_paged_block_bytes(int format, int page_size, int d);

/*
 * Appends new K and V rows to the cache, rotated by their positions on the
 * way, and rotates Q rows with them.
 *   k, v   : in,  bf16, element (row, head, i) at row * x_row + head * x_head + i
 *            with Hkv heads (strides in elements, multiples of 8: rows as a
 *            fused projection leaves them need no copy)
 *   cu_new : in,  int [B + 1]
 *   rows   : rows of the tensors (cu_new[B] at least)
 *   q      : in,  as k with H heads, or NULL: no Q
 *   q_out  : out, bf16 [rows, H, d]; padding rows are left as they were
 *   rope   : in,  fp32 [rope_len, rot]: row p holds cos of the rot/2 angles of
 *            position p, then their sines; NULL with rot = 0: no rotation
 *   rot    : elements of a row that are rotated, a multiple of 16 up to d.
 *            x'_a = x_a cos - x_b sin, x'_b = x_b cos + x_a sin with (a, b) =
 *            (i, i + rot/2), or, interleaved = 1, (2i, 2i + 1); in fp32, each
 *            product and sum rounded
 * K and Q are rotated, V is not.  bf16 caches take the results rounded once.
 * 4-bit caches take, with y = x / g in fp32 and per 16 elements, the scale
 * s = e4m3(max |y| / 6) (at most 448) and the codes e2m1(y / s), to nearest,
 * ties to even; a negative zero becomes zero, a scale that rounds to 0 stores
 * zeros, a block with an infinity or a NaN reads back as NaN.
 */
int fa_paged_append(const fa_paged_cache* cache, const void* k, long long k_row, long long k_head,
                    const void* v, long long v_row, long long v_head, const int* cu_new, int rows,
                    const void* q, long long q_row, long long q_head, void* q_out, int H,
                    const float* rope, int rope_len, int rot, int interleaved, void* stream);

/*
 * Reads the last rows of each sequence out of the cache as bf16 (the rotated
 * rows that fa_paged_append wrote, 4-bit values rounded once).
 *   cu_new, rows : as fa_paged_append
 *   k, v         : out, bf16 [rows, Hkv, d]; a row without a usable place is
 *                  zeros, padding rows are left as they were
 */
int fa_paged_read(const fa_paged_cache* cache, const int* cu_new, int rows, void* k, void* v,
                  void* stream);

/*
 * Attention of each sequence's last rows over its cached positions, its own
 * included (append first).  The row at position p sees the positions j <= p
 * with p - j < window, and the positions j < sinks (j <= p):
 *   O = softmax(scale q K^T) V over these, LSE as fa_fwd.
 * Positions on a page outside the cache count as masked (FA_ERR_INVALID_ARG is
 * recorded).  A row that sees nothing (a sequence of length 0, or longer than its
 * pages, which is recorded) gets O = 0, LSE = -inf.
 *   q        : in,  bf16 with H heads, strides as fa_paged_append; query head
 *              h reads key head h / (H / Hkv)
 *   o        : out, bf16 [rows, H, d]; lse: out, fp32 [rows, H]; padding rows
 *              are left as they were
 *   max_new  : rows of a sequence at most (1 for a decode step); rows beyond
 *              it are not computed and FA_ERR_INVALID_ARG is recorded
 *   H        : query heads, a multiple of Hkv
 *   window   : positions that a row sees, itself included; 0 = all before it
 *   sinks    : first positions that every row sees besides
 *   workspace: fa_fwd_paged_workspace_bytes() bytes on the current device,
 *              256-byte aligned, contents on entry irrelevant
 * What positions outside every row's sight hold (the rest of a page, too) does
 * not matter, infinities and NaN included, and the page table's entries of pages
 * without a position in sight are not looked at: such pages may be given
 * back as a window moves on.  A position that some row of the same call
 * sees must be finite where another does not see it.
 * The work does not depend on how lengths are spread over sequences; cached
 * rows are read once for every 16 (row, query head of the group) pairs, so
 * long chunks of new rows are served, but prompts better by fa_fwd_window.
 */
size_t fa_fwd_paged_workspace_bytes(int d);
int fa_fwd_paged(const fa_paged_cache* cache, const void* q, long long q_row, long long q_head,
                 void* o, float* lse, const int* cu_new, int rows, int max_new, int H, float scale,
                 int window, int sinks, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, then returns and clears the device status word:
 * FA_OK, or FA_ERR_TIMEOUT when a kernel gave up on a bounded wait since the
 * last call, or FA_ERR_INVALID_ARG when a kernel of the paged cache or of packed
 * sequences met tables that it could not follow, or FA_ERR_CUDA when the synchronisation itself failed.
 */
int fa_last_device_status(void* stream);

/* Extra detail about the last device status: the code of the wait site that
 * timed out or of the check that failed (0 if none).  Valid after fa_last_device_status(). */
int fa_last_device_site(void);

/* Human-readable name of a fa_status value (static string). */
const char* fa_status_string(int status);

/*
 * Diagnostic: evaluates the kernels' polynomial exp2 (the software-emulated
 * exponential on the FMA pipe, FlashAttention-4 abstract item 2; "Программная
 * эмуляция экспоненты" of "FlashAttention-3 и FlashAttention-4") on n fp32
 * values.  x, y are device pointers; the input is clamped to the kernels'
 * domain [-125, 127] first.  For testing the approximation only.
 */
int fa_exp2_poly_eval(const float* x, float* y, long long n, void* stream);

/*
 * Diagnostic: runs one kernel whose only work is an mbarrier wait that nothing
 * ever completes, bounded by limit_ns nanoseconds (1 ms .. 10 s).  It returns
 * through the same give-up path as the attention kernels, so a following
 * fa_last_device_status() must report FA_ERR_TIMEOUT and the CUDA context
 * stays usable.  For testing the bounded-wait machinery without a fault.
 */
int fa_debug_bounded_wait(unsigned long long limit_ns, void* stream);

/*
 * Timing of the main kernels.  fa_timing_enable(1) makes every later fa_fwd /
 * fa_bwd record a pair of CUDA events on its stream around its main kernel
 * (the forward kernel; the backward main kernel, between the pre- and
 * post-processing kernels); fa_timing_enable(0) stops it.  The events belong
 * to the library (created on first use on the current device).
 * fa_timing_last_ms(kernel, &ms) waits for the last recorded pair of that
 * kernel (0 = forward, 1 = backward main) and returns its elapsed time in
 * milliseconds; FA_ERR_INVALID_ARG if none was recorded.
 */
int fa_timing_enable(int enable);
int fa_timing_last_ms(int kernel, float* ms);

/*
 * Number of kernels the library has launched since it was loaded, over all
 * entry points, streams and threads (launches that CUDA refused are not
 * counted).  The difference of two readings counts the launches in between,
 * e.g. in a timed region: fa_fwd launches one kernel, or two when it splits
 * its last partial round of work in the caller's workspace (the forward,
 * then the merge); fa_bwd three;
 * fa_bwd_deterministic three; fa_fwd_fp8 three (two preparation kernels and
 * the forward; four with the merge, as fa_fwd); fa_fwd_splitkv two;
 * fa_fwd_2cta one; fa_bwd_2cta three; fa_fwd_window one; fa_bwd_window three;
 * fa_paged_append and fa_paged_read one; fa_packed_plan and fa_rotate one,
 * fa_fwd_packed one, or two when it cuts items into key ranges, fa_bwd_packed three;
 * fa_fwd_paged two (the forward, then the join of segments that several CTAs
 * shared).
 */
unsigned long long fa_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
