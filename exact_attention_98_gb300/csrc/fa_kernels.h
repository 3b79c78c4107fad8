// Parameter blocks and launchers shared between the C-ABI layer (fa_api.cu)
// and the kernel translation units (fa_fwd.cu, fa_bwd.cu).  Host code only
// sees these declarations; the kernels are internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "fa_fastdiv.h"

namespace fa {

// Tile shape shared by the forward and backward kernels: 128 query rows x 128
// key rows per step, the tcgen05 M = 128 single-CTA shape.
constexpr int kBlockM = 128;
constexpr int kBlockN = 128;
// Conditional-rescale threshold, in log2 units of the scaled scores: O and the
// row sum are rescaled only when a row max grows by more than a factor 2^2.
// In exact arithmetic any value gives the same result (the final division
// uses the same stale max).  In bf16 it matters: P is rounded to bf16 for the
// P V product, and under a stale reference max the dominant weight of a row
// is some value in [1, 2^tau) instead of exactly 1, so its rounding error
// reaches O.  A CPU emulation of the tiled algorithm on the softmax-stress
// inputs gave a worst O error of 0.64x the tolerance at tau = 2 and 1.22x at
// tau = 8; on N(0,1) inputs tau = 2 rescales about 0.7% of row-tiles.
constexpr float kRescaleThreshold = 2.0f;

struct FwdParams {
  CUtensorMap tm_q;  // bf16 [BH, N, d], box {64, 128, 1}, 128B swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_o;      // bf16 O [BH, N, d], box {64, 128, 1}, 128B swizzle (bulk stores)
  void* o;               // bf16 [BH, N, d]
  float* lse;            // fp32 [BH, N]
  unsigned int* status;  // device status word
  int N;
  int BH;
  int n_qblk;   // ceil(N / 256): a work item is two 128-row query tiles (pair: see below)
  int n_items;  // n_qblk * BH * num_splits
  // Split-KV: work items from block split_from on cut their key tiles into
  // num_splits contiguous ranges, one item each; such an item writes O
  // normalised over its range and its LSE (fp32) to the partial buffers, slot
  // part = (block - split_from) * num_splits + range, 256 rows per slot:
  // o_part [slots, 256, d], lse_part [slots, 256].  A merge kernel combines
  // the ranges.  split_from = number of blocks: no split, o_part unused.
  int split_from;
  int num_splits;
  float* o_part;
  float* lse_part;
  // FP8 inputs (fp8 != 0): tm_q, tm_k, tm_v map the e4m3 Q, K and V^T of
  // Fp8Buffers; scores carry the row's Q and the head's K descale, O the
  // head's V descale.
  int fp8;
  const float* q_descale;       // [BH, N]
  const unsigned int* fp8_amax;  // [2 * BH]: K then V amax per head (fp32 bits)
  // Pair mode (pair != 0; bf16, d = 128, no split): clusters of two CTAs
  // share each product (M = 256); a work item is 512 query rows, n_qblk =
  // ceil(N / 512), and tm_k's box is 64 rows (each CTA loads half of a K
  // tile).
  int pair;
  int causal;
  float c;          // scale * log2(e): scores enter exp2 in these units
  float ln2;        // ln(2), to turn the log2-unit row max into LSE
  int poly_per_octet;  // exponentials per 8 on the FMA pipe (0..3)
  // BH, n_qblk and num_splits as multiply-shift divisors for the work-item
  // walk that every role of every CTA repeats per item
  FastDiv div_bh, div_qblk, div_splits;
  // Sliding window (window > 0; bf16, no split): a row sees the `window` keys up
  // to itself and the first `sinks` keys.  tm_k and tm_v have B * Hkv slices;
  // query head h reads key head div_group(h).  A work item is two
  // query tiles of one head (win_tiles = 2), or one query tile of two heads (1);
  // n_qblk = ceil(N / (128 win_tiles)), div_bh's divisor the items of one
  // query block.
  int window;
  int sinks;
  int win_tiles;
  FastDiv div_group;
};

// Default share of the forward's exponentials evaluated by the polynomial on
// the FMA pipe (per 8); FA_FWD_POLY_PER_OCTET in the environment selects
// another pre-built instantiation (0..3).
constexpr int kDefaultPolyPerOctet = 0;

struct BwdParams {
  CUtensorMap tm_q;   // bf16 [BH, N, d]
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_do;
  // fp32 dQ target, box {16, 128, 1}, 64B swizzle: the accumulator
  // [BH, N, d] (or, with dq_part, the per-key-tile slices [n_kblk * BH, N, d])
  CUtensorMap tm_dq;
  // bf16 dK and dV [BH, N, d], box {64, 128, 1}, 128B swizzle (bulk stores)
  CUtensorMap tm_dk;
  CUtensorMap tm_dv;
  const float* lse;   // fp32 [BH, N]
  const float* dsum;  // fp32 [BH, N]: D = rowsum(dO * O)
  float* dq_acc;      // fp32 [BH, N, d], zeroed before the main kernel (atomic mode)
  // Per-key-tile dQ contributions (key tile kt of head bh would write
  // dq_part[kt * BH + bh] with plain stores instead of reducing): no entry
  // point sets it any more (nullptr; the deterministic mode has its own dQ
  // kernel).  The drains' store branches that read it stay because the
  // kernel measured 1-2% slower without them (code layout).
  float* dq_part;     // fp32 [n_kblk * BH, N, d]
  void* dk;           // bf16 [BH, N, d]
  void* dv;           // bf16 [BH, N, d]
  unsigned int* status;
  int N;
  int BH;
  int n_kblk;  // ceil(N / 128)
  int causal;
  float c;      // scale * log2(e)
  float scale;  // applied to dK in the write-out and to dQ in its conversion (dS leaves it out)
  float inv_scale;  // 1 / scale: -LSE / scale is the bias in raw score units
  float log2e;
  // Sliding window (the window kernel only): a row sees the `window` keys up to
  // itself (window <= N); `group` query heads share a key head, and K, V, dK,
  // dV and BH are of the key heads.  With sink_main, the fp32 dV and
  // (unscaled) dK of the first `sinks` keys go there, [BH, 2 (dK, dV),
  // sink_rows, d], to be joined with what the first tokens get from
  // queries whose windows have left them (fa_window.cu).
  int window;
  int group;
  int sinks;
  int sink_rows;
  float* sink_main;
  // Items (key tile of a key head) from split_from on are cut into split_parts
  // parts, whose fp32 dK (unscaled) and dV go to tile_part [part, 2, 128, d].
  int split_from;
  int split_parts;
  float* tile_part;
  FastDiv div_kblk, div_parts;  // window: by n_kblk, by split_parts
};

// What the sliding-window backward does beside its main kernel (fa_window.cu):
// D and the start of the dQ accumulator before it, the first tokens' dK and dV
// after it.
struct WindowParams {
  const __nv_bfloat16* q;  // [BHkv * group, N, d]
  const __nv_bfloat16* k;  // [BHkv, N, d]
  const __nv_bfloat16* v;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  const float* lse;   // [BHkv * group, N]
  float* dsum;        // [BHkv * group, N]
  float* dq_acc;      // [BHkv * group, N, d]
  __nv_bfloat16* dq;
  float* sink_part;   // [slots + 1, BHkv, 2 (dK, dV), sink_rows, d]; the last slot is the main kernel's
  const float* tile_part;  // the main kernel's split items (BwdParams)
  int split_from, split_parts, n_kblk;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int N;
  int BHkv;
  int group;
  int window;
  int sinks;
  int sink_rows;  // sinks rounded up to 16
  int slots;      // parts that the rows of a key head's queries are cut into
  int slot_rows;  // rows of a part, a multiple of 16
  FastDiv div_tiles, div_last_tiles;  // by the 16-row tiles of a part, of the last part
  unsigned int* status;
  float c;        // scale * log2(e)
  float log2e;
  float scale;
  int sink_blocks, tile_blocks;  // set by launch_window_post
};

// Backward by CTA pairs (d = 128): a cluster of two CTAs owns two
// consecutive key tiles of one head (256 keys) and shares every product as
// one tcgen05 cta_group::2 MMA.
struct BwdPairParams {
  CUtensorMap tm_q;     // bf16 [BH, N, d], box {64, 128, 1}: Q rows x one 64-column half of d
  CUtensorMap tm_do;
  CUtensorMap tm_q64;   // box {64, 64, 1}: this CTA's 64 query rows, one 64-column block
  CUtensorMap tm_do64;
  CUtensorMap tm_k;     // box {64, 128, 1}
  CUtensorMap tm_v;
  const float* lse;     // fp32 [BH, N]
  const float* dsum;    // fp32 [BH, N]: D = rowsum(dO * O)
  float* dq_acc;        // fp32 [BH, N, d], zeroed before the main kernel
  void* dk;             // bf16 [BH, N, d]
  void* dv;             // bf16 [BH, N, d]
  unsigned int* status;
  int N;
  int BH;
  int n_kblk;   // ceil(N / 128)
  int n_kpair;  // ceil(n_kblk / 2): key-tile pairs per head
  int causal;
  float c;          // scale * log2(e)
  float scale;      // applied to dK in the write-out and to dQ in its conversion
  float inv_scale;
};

// Backward main kernel run by CTA pairs (d = 128 only).
cudaError_t launch_bwd_pair(const BwdPairParams& p, cudaStream_t stream);

// FP8 forward inputs (d = 128), in the caller's workspace.
struct Fp8Buffers {
  uint8_t* q8;          // e4m3 [BH, N, 128], Q rotated, one scale per row
  float* q_descale;     // [BH, N]: amax / 448 of each rotated Q row
  uint8_t* k8;          // e4m3 [BH, N, 128], K rotated, one scale per head
  uint8_t* v8t;         // e4m3 [BH, 128, Np], V transposed, one scale per head
  unsigned int* amax;   // [2 * BH]: fp32 bits of the K amax per head, then V
  float* amax_part;     // [2, BH, ceil(N / 128)]: K, then V amax of each 128-row block
  int Np;               // N rounded up to a multiple of 16 (V^T row pitch)
};
// Number of floats of Fp8Buffers::amax_part.
size_t fp8_amax_part_count(int BH, int N);
// The bf16 inputs of the FP8 preparation: [BH, N, d] maps as the forward's
// (box {64, 128, 1}, 128-byte swizzle).
struct Fp8Maps {
  CUtensorMap q;
  CUtensorMap k;
  CUtensorMap v;
};
// Rotation (optional) and quantisation of Q, K, V into `b`; bounded waits
// report through `status`.
cudaError_t launch_fp8_prepare(const Fp8Maps& maps, const Fp8Buffers& b, int BH, int N, int rotate,
                               unsigned int* status, cudaStream_t stream);

// Launches `kernel` on `stream` as a programmatic dependent launch: it may
// start (allocate, initialise its barriers, set up tensor memory) while the
// kernel before it in the stream is finishing, and it calls
// grid_dependency_wait() before it reads or writes anything that kernel, or
// any earlier work in the stream, produces or consumes.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Number of SMs of the current device (0 on an error); looked up once per device.
int sm_count();

// Raises Kernel's limit of dynamic shared memory on the current device, and
// refuses a build whose register count differs from `regs` (0: any): a
// setmaxnreg split assumes the launch allocation, and an over-committed one
// would never finish.  Asks the runtime once per device.
template <auto* Kernel>
cudaError_t configure_kernel(int smem, int regs = 0) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if (regs > 0) {
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, Kernel);
    if (err != cudaSuccess) return err;
    if (attr.numRegs != regs) return cudaErrorInvalidConfiguration;
  }
  err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return err;
}

// The launch wrappers end with `return launched(n)`: the launch error of the
// n kernels just launched, which are added to the library's launch count
// (fa_launch_count) when there is none.
cudaError_t launched(unsigned int n);

// Forward: one launch of the tcgen05 kernel for head dim d (64 or 128).
cudaError_t launch_fwd(const FwdParams& p, int d, cudaStream_t stream);
// Split-KV merge of the split blocks of `p`: LSE = ln sum_s exp(LSE_s),
// O = sum_s exp(LSE_s - LSE) O_s -> bf16 O and fp32 LSE.
cudaError_t launch_fwd_merge(const FwdParams& p, void* o, float* lse, int d, cudaStream_t stream);

// Backward: D = rowsum(dO * O) and dQ accumulator zeroing.
cudaError_t launch_bwd_pre(const void* o, const void* dout, float* dsum, float* dq_acc,
                           long long rows, int d, cudaStream_t stream);
// Backward main kernel (key/value stationary).
cudaError_t launch_bwd_main(const BwdParams& p, int d, cudaStream_t stream);
// The same kernel with a sliding window and shared key heads (p.window, p.group).
cudaError_t launch_bwd_window(const BwdParams& p, int d, cudaStream_t stream);
cudaError_t launch_bwd_window64(const BwdParams& p, cudaStream_t stream);  // its d = 64 form (fa_bwd_window64.cu)
// Before it, where queries see first tokens that their windows have left: D, and
// those pairs' share of dQ in the accumulator, of dK and dV in sink_part.
cudaError_t launch_window_pre(const WindowParams& p, int d, cudaStream_t stream);
// After it: dQ as bf16, and the first tokens' dK and dV rows and those of split
// items from all their parts.
cudaError_t launch_window_post(WindowParams p, int d, cudaStream_t stream);
// The same kernel computing dK and dV only (p.tm_dq, p.dq_acc and p.dq_part
// unused): the deterministic mode's first pass.
cudaError_t launch_bwd_dkdv(const BwdParams& p, int d, cudaStream_t stream);
// dQ = mul * dQ accumulator -> bf16 (mul: the softmax scale, which the main
// kernels leave out of dS).
cudaError_t launch_bwd_post(const float* dq_acc, void* dq, long long elems, float mul,
                            cudaStream_t stream);

// The paged key/value cache as the kernels see it (fa_paged_cache in fa.h).
struct PagedView {
  uint8_t* pages;        // [num_pages, Hkv] blocks (see fa_paged.cuh)
  const int* page_table;  // [B, max_pages]
  const int* seq_lens;    // [B]
  const float* k_scale;   // [Hkv], or null: 1
  const float* v_scale;
  int B;
  int Hkv;
  int num_pages;
  int page_shift;  // log2(page_size)
  int max_pages;
};

struct PagedAppendParams {
  PagedView c;
  const int* cu;  // [B + 1]: rows of sequence b are cu[b] .. cu[b+1]-1
  int rows;
  int tokens;  // rows a block of threads takes (set by the launcher)
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;  // null: no Q to rotate
  __nv_bfloat16* q_out;    // [rows, H, d]
  long long k_row, k_head, v_row, v_head, q_row, q_head;  // strides in elements
  int H;
  const float* rope;  // [rope_len, rot]: rot/2 cosines, then rot/2 sines
  int rope_len;
  int rot;  // 0: no rotation
  int interleaved;
  FastDiv div_q, div_kv;  // rows of a token: H (1 without Q), 2 Hkv
  unsigned int* status;
};

struct PagedReadParams {
  PagedView c;
  const int* cu;
  int rows;
  int tokens;
  __nv_bfloat16* k;  // [rows, Hkv, d]
  __nv_bfloat16* v;
  FastDiv div_heads;  // 2 Hkv (rows of a token)
  unsigned int* status;
};

cudaError_t launch_paged_append(PagedAppendParams p, int d, bool fp4, cudaStream_t stream);
cudaError_t launch_paged_read(PagedReadParams p, int d, bool fp4, cudaStream_t stream);

struct FwdPagedParams {
  CUtensorMap tm;  // bf16 cache: (d, page_size, num_pages * Hkv * 2), box {64, 16, 1}
  PagedView c;
  const int* cu;
  int rows;
  int max_new;  // rows of a sequence at most
  const __nv_bfloat16* q;
  long long q_row, q_head;
  __nv_bfloat16* o;  // [rows, H, d]
  float* lse;        // [rows, H]
  int H;
  int group;   // H / Hkv
  int window;  // INT_MAX: none
  int sinks;
  float scale;  // times log2(e): scores enter exp2 in these units
  // workspace: two partial slots per worker (a warp) of a block's rows each, and
  // where worker i's last segment goes on
  float* part_o;   // [2 * workers, rows of a block, d], not normalised
  float* part_ml;  // [2 * workers, 2, rows of a block]: references in log2 units, row sums
  int4* info;      // [workers]: {parts, sequence, key head * blocks of rows + block, 0}
  unsigned int* status;
};

// Warps of the paged forward at most, per SM and on the current device (0 on an
// error), and rows of a block at most: its workspace.
constexpr int kPagedWorkersPerSm = 12;
constexpr int kPagedRows = 16;
int fwd_paged_workers();
// One launch of the forward and one of the join of its split segments.
cudaError_t launch_fwd_paged(const FwdPagedParams& p, int d, bool fp4, long long max_units,
                             cudaStream_t stream);

}  // namespace fa
