// C ABI of libfa.so: argument validation, TMA descriptor encoding, launches,
// the device status word, and two small diagnostic kernels.  The operations
// and their argument conventions are documented in include/fa.h.
#include <math.h>
#include <stdlib.h>
#include <atomic>
#include <mutex>
#include <stdint.h>

#include "fa.h"
#include "fa_device.cuh"
#include "fa_bwd_dq.h"
#include "fa_kernels.h"
#include "fa_packed.cuh"
#include "fa_paged.cuh"

namespace fa {

// The status word every kernel writes through a pointer (see fa_device.cuh).
__device__ unsigned int g_status_word;

// Kernels launched by this library since it was loaded (fa_launch_count).
std::atomic<unsigned long long> g_launches{0};

cudaError_t launched(unsigned int n) {
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) g_launches.fetch_add(n, std::memory_order_relaxed);
  return err;
}

// Number of SMs of the current device (the persistent forward's grid).
int sm_count() {
  static std::mutex mu;
  static int counts[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (counts[dev] == 0 &&
      cudaDeviceGetAttribute(&counts[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    counts[dev] = 0;
  return counts[dev];
}

namespace {

int g_last_site = 0;

// Optional event pairs around the main kernels (kernel 0 = forward, 1 =
// backward main), recorded on the launch stream when timing is enabled.
struct KernelTiming {
  std::mutex mu;
  bool enabled = false;
  cudaEvent_t start[2] = {nullptr, nullptr};
  cudaEvent_t stop[2] = {nullptr, nullptr};
  bool recorded[2] = {false, false};
};
KernelTiming g_timing;


cudaError_t timing_record(int kernel, bool at_start, cudaStream_t s) {
  std::lock_guard<std::mutex> lock(g_timing.mu);
  if (!g_timing.enabled) return cudaSuccess;
  cudaEvent_t& ev = at_start ? g_timing.start[kernel] : g_timing.stop[kernel];
  if (!ev) {
    cudaError_t e = cudaEventCreate(&ev);
    if (e != cudaSuccess) return e;
  }
  if (!at_start) g_timing.recorded[kernel] = true;
  return cudaEventRecord(ev, s);
}

// Device address of g_status_word for the current device, looked up once per
// device with that device current.
unsigned int* status_ptr() {
  static std::mutex mu;
  static unsigned int* ptrs[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<unsigned int*>(p);
  }
  return ptrs[dev];
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// bf16 [BH, N, d] viewed as a 3-D tensor (d, N, BH); the box is 64 columns
// (128 bytes, one 128B-swizzle row) x box_rows rows x 1 head.  Rows past N
// read as zeros.
bool encode_tile_map(CUtensorMap* map, const void* base, int N, int BH, int d,
                     unsigned int box_rows = 128) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of packed sequences (fa_rows), bf16, viewed as (d, rows, heads): box as
// encode_tile_map.  A single row's or head's stride does not matter.
bool encode_rows_map(CUtensorMap* map, const fa_rows& t, int rows, int heads, int d,
                     unsigned int box_rows = kBlockM) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(rows > 1 ? t.row : d) * 2,
                                 static_cast<cuuint64_t>(heads > 1 ? t.head : d) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.data, dims, strides, box, elem_strides,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 8-bit [slices, rows, cols] tensor, rows of `pitch` bytes, box 128 x 128:
// one 128-byte swizzle row per tile row (the FP8 forward's e4m3 operands).
bool encode_u8_map(CUtensorMap* map, const void* base, long long cols, long long rows,
                   long long slices, long long pitch) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(slices)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch),
                                 static_cast<cuuint64_t>(pitch) * static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[3] = {128, 128, 1};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
            elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Share of the forward's exponentials on the FMA pipe, per 8: the initial
// value from FA_FWD_POLY_PER_OCTET (default kDefaultPolyPerOctet), then
// whatever fa_set_exp2_poly_share() sets.
std::atomic<int>& poly_share() {
  static std::atomic<int> value{[] {
    const char* e = getenv("FA_FWD_POLY_PER_OCTET");
    if (e && e[0] >= '0' && e[0] <= '3' && e[1] == '\0') return e[0] - '0';
    return kDefaultPolyPerOctet;
  }()};
  return value;
}

// fp32 [slices, N, d] viewed as (d, N, slices), slices = BH (the dQ
// accumulator) or n_kblk * BH (the deterministic mode's per-key-tile
// contributions); box 16 columns (64 bytes) x 128 rows x 1 slice with 64-byte
// swizzle, for bulk reduce-adds and stores.  Rows past N are dropped by the
// TMA unit.
bool encode_dq_map(CUtensorMap* map, const float* base, int N, long long slices, int d) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(slices)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4,
                                 static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 4};
  const cuuint32_t box[3] = {16, 128, 1};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box,
            elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shape checks shared by forward and backward.  Returns FA_OK, or the error,
// with *empty set when there is nothing to compute.
int check_shape(int B, int H, int N, int d, float scale, bool* empty) {
  *empty = false;
  if (B < 0 || H < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || N == 0) {
    *empty = true;
    return FA_OK;
  }
  const long long bh = static_cast<long long>(B) * H;
  // grid sizes and int row indices inside the kernels
  if (bh > (1LL << 30) || static_cast<long long>(N) * bh > (1LL << 40)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

constexpr int kMaxSinks = 128;  // first tokens of a sliding window: one key tile
constexpr size_t kWsAlign = 256;
size_t round_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

__global__ void exp2_poly_eval_kernel(const float* x, float* y, long long n) {
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x)
    y[i] = exp2_poly(x[i]);
}

// One mbarrier that nothing arrives on; the bounded wait must give up.  One
// warp waits in the warp-uniform form the forward's MMA-issuing warp uses
// (every lane waits, the result is voted), so its give-up path is the one
// exercised.
__global__ void bounded_wait_kernel(unsigned int* status, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t mbar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(smem_u32(&mbar), 1);
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl ctl{&abort_flag, status};
  mbar_wait_warp(smem_u32(&mbar), 0, ctl, 0x0F0, limit_ns);
  __syncthreads();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_TOO_LARGE: return "FA_ERR_TOO_LARGE";
    default: return "FA_ERR_UNKNOWN";
  }
}

namespace {

int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
             int d, float scale, int causal, int num_splits, void* workspace,
             size_t workspace_bytes, void* stream, int fp8 = 0, int rotate = 0, int pair = 0);

// Partial buffers of `slots` split items of 256 rows: O (fp32, d columns),
// then LSE.
size_t split_scratch_bytes(size_t slots, int d) {
  return round_up(slots * 2 * kBlockM * d * sizeof(float)) +
         round_up(slots * 2 * kBlockM * sizeof(float));
}

// The forward's last-round split.  Non-causal items all cost the same, so
// when they do not fill whole rounds of the persistent grid (one CTA per SM)
// the last partial round's `tail` blocks are cut into `ns` key ranges, as
// many as fill that round, each of at least 8 key tiles.  False when no
// split applies.
bool tail_split(long long blocks, int n_ktiles, int causal, int sms, int* tail, int* ns) {
  if (causal || sms <= 0 || blocks <= sms) return false;
  const int t = static_cast<int>(blocks % sms);
  if (t == 0) return false;
  const int n = sms / t;
  if (n < 2 || n_ktiles < 8 * n) return false;
  *tail = t;
  *ns = n;
  return true;
}

// Scratch of the last-round split of a (B, H, N, d) forward on the current
// device; 0 when none applies.
size_t tail_split_bytes(int B, int H, int N, int d, int causal) {
  const long long blocks = static_cast<long long>(B) * H * ((N + 2 * kBlockM - 1) / (2 * kBlockM));
  int tail = 0, ns = 0;
  if (!tail_split(blocks, (N + kBlockN - 1) / kBlockN, causal, sm_count(), &tail, &ns)) return 0;
  return split_scratch_bytes(static_cast<size_t>(tail) * ns, d);
}

// Bytes of the FP8 operands and scales at the head of the FP8 workspace.
size_t fp8_buffer_bytes(int B, int H, int N) {
  const size_t BH = static_cast<size_t>(B) * H;
  const size_t rows = BH * N;
  const size_t Np = (static_cast<size_t>(N) + 15) / 16 * 16;
  return 2 * round_up(rows * 128) + round_up(BH * 128 * Np) + round_up(rows * sizeof(float)) +
         round_up(2 * BH * sizeof(unsigned int)) +
         round_up(fp8_amax_part_count(static_cast<int>(BH), N) * sizeof(float));
}

}  // namespace

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
           int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, N, d, scale, causal, 1, workspace, workspace_bytes,
                  stream);
}

size_t fa_fwd_workspace_bytes(int B, int H, int N, int d, int causal) {
  bool empty = false;
  if (check_shape(B, H, N, d, 1.0f, &empty) != FA_OK || empty) return 0;
  return tail_split_bytes(B, H, N, d, causal);
}

int fa_fwd_2cta(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int N, int d, float scale, int causal, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, N, d, scale, causal, 1, nullptr, 0, stream, 0, 0, 1);
}

size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int N, int d, int num_splits) {
  bool empty = false;
  if (check_shape(B, H, N, d, 1.0f, &empty) != FA_OK || empty) return 0;
  if (num_splits < 2) return 0;
  const size_t blocks = static_cast<size_t>(B) * H * ((N + 2 * kBlockM - 1) / (2 * kBlockM));
  return split_scratch_bytes(blocks * num_splits, d);
}

size_t fa_fwd_fp8_workspace_bytes(int B, int H, int N, int d) {
  bool empty = false;
  if (check_shape(B, H, N, d, 1.0f, &empty) != FA_OK || empty || d != 128) return 0;
  return fp8_buffer_bytes(B, H, N) + tail_split_bytes(B, H, N, d, 0);
}

int fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int N, int d, float scale, int causal, int rotate, void* workspace,
               size_t workspace_bytes, void* stream) {
  if (rotate != 0 && rotate != 1) return FA_ERR_INVALID_ARG;
  return fwd_impl(q, k, v, o, lse, B, H, N, d, scale, causal, 1, workspace, workspace_bytes, stream,
                  1, rotate);
}

int fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                   int N, int d, float scale, int causal, int num_splits, void* workspace,
                   size_t workspace_bytes, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, N, d, scale, causal, num_splits, workspace,
                  workspace_bytes, stream);
}

int fa_set_exp2_poly_share(int per_octet) {
  if (per_octet < 0 || per_octet > 3) return FA_ERR_INVALID_ARG;
  poly_share().store(per_octet, std::memory_order_relaxed);
  return FA_OK;
}

int fa_get_exp2_poly_share(void) { return poly_share().load(std::memory_order_relaxed); }

namespace {

// num_splits > 1: every block cut into that many key ranges (fa_fwd_splitkv,
// workspace required).  fp8: the workspace holds the e4m3 operands first.
// Otherwise the workspace is optional and, when given, takes the last-round
// split's partials (after the FP8 buffers in FP8 mode).
int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
             int d, float scale, int causal, int num_splits, void* workspace,
             size_t workspace_bytes, void* stream, int fp8, int rotate, int pair) {
  bool empty = false;
  int rc = check_shape(B, H, N, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse))
    return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  const int n_ktiles = (N + kBlockN - 1) / kBlockN;
  if (num_splits < 1 || num_splits > n_ktiles) return FA_ERR_INVALID_ARG;
  if ((fp8 || pair) && d != 128) return FA_ERR_UNSUPPORTED;
  // the FP8 preparation counts its work units (three per 128-row block of a
  // head) in int
  if (fp8 && static_cast<long long>(B) * H * (3LL * ((N + 127) / 128) + 1) > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (num_splits > 1 || fp8 || workspace != nullptr) {
    const size_t need = fp8 ? fa_fwd_fp8_workspace_bytes(B, H, N, d)
                        : num_splits > 1 ? fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits)
                                         : fa_fwd_workspace_bytes(B, H, N, d, causal);
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0) return FA_ERR_WORKSPACE;
  }

  FwdParams p = {};
  const int BH = B * H;
  const long long rows = static_cast<long long>(BH) * N;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.fp8 = fp8;
  p.q_descale = nullptr;
  p.fp8_amax = nullptr;
  // the part of the workspace the last-round split may use
  char* split_ws = static_cast<char*>(workspace);
  if (fp8) {
    Fp8Buffers fb;
    char* w = static_cast<char*>(workspace);
    fb.Np = (N + 15) / 16 * 16;
    fb.q8 = reinterpret_cast<uint8_t*>(w);
    w += round_up(static_cast<size_t>(rows) * 128);
    fb.k8 = reinterpret_cast<uint8_t*>(w);
    w += round_up(static_cast<size_t>(rows) * 128);
    fb.v8t = reinterpret_cast<uint8_t*>(w);
    w += round_up(static_cast<size_t>(BH) * 128 * fb.Np);
    fb.q_descale = reinterpret_cast<float*>(w);
    w += round_up(static_cast<size_t>(rows) * sizeof(float));
    fb.amax = reinterpret_cast<unsigned int*>(w);
    w += round_up(2 * static_cast<size_t>(BH) * sizeof(unsigned int));
    fb.amax_part = reinterpret_cast<float*>(w);
    split_ws = static_cast<char*>(workspace) + fp8_buffer_bytes(B, H, N);
    if (!encode_u8_map(&p.tm_q, fb.q8, 128, N, BH, 128) ||
        !encode_u8_map(&p.tm_k, fb.k8, 128, N, BH, 128) ||
        !encode_u8_map(&p.tm_v, fb.v8t, fb.Np, 128, BH, fb.Np))
      return FA_ERR_CUDA;
    Fp8Maps maps;
    if (!encode_tile_map(&maps.q, q, N, BH, d) || !encode_tile_map(&maps.k, k, N, BH, d) ||
        !encode_tile_map(&maps.v, v, N, BH, d))
      return FA_ERR_CUDA;
    unsigned int* status = status_ptr();
    if (!status) return FA_ERR_CUDA;
    if (launch_fp8_prepare(maps, fb, BH, N, rotate, status, s) != cudaSuccess) return FA_ERR_CUDA;
    p.q_descale = fb.q_descale;
    p.fp8_amax = fb.amax;
  } else if (!encode_tile_map(&p.tm_q, q, N, BH, d) ||
             !encode_tile_map(&p.tm_k, k, N, BH, d, pair ? 64 : 128) ||
             !encode_tile_map(&p.tm_v, v, N, BH, d)) {
    return FA_ERR_CUDA;
  }
  if (!encode_tile_map(&p.tm_o, o, N, BH, d)) return FA_ERR_CUDA;
  p.o = o;
  p.lse = lse;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = N;
  p.BH = BH;
  p.pair = pair;
  const int item_rows = (pair ? 4 : 2) * kBlockM;
  p.n_qblk = (N + item_rows - 1) / item_rows;
  p.causal = causal;
  p.c = scale * 1.4426950408889634f;
  p.ln2 = 0.6931471805599453f;
  p.poly_per_octet = poly_share().load(std::memory_order_relaxed);
  if (static_cast<long long>(p.n_qblk) * BH * num_splits > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const int blocks = p.n_qblk * BH;
  // Which blocks are split: all of them (num_splits > 1), else, when the
  // caller gave a workspace, the last partial round of the persistent grid
  // (see tail_split); the partials go to the workspace.
  p.split_from = blocks;
  p.num_splits = 1;
  p.o_part = p.lse_part = nullptr;
  int tail = 0, ns = 0;
  if (num_splits > 1) {
    p.split_from = 0;
    p.num_splits = num_splits;
  } else if (workspace != nullptr && !pair &&
             tail_split(blocks, n_ktiles, causal, sm_count(), &tail, &ns)) {
    p.split_from = blocks - tail;
    p.num_splits = ns;
  }
  if (p.split_from < blocks) {
    const size_t slots = static_cast<size_t>(blocks - p.split_from) * p.num_splits;
    p.o_part = reinterpret_cast<float*>(split_ws);
    p.lse_part = reinterpret_cast<float*>(split_ws + round_up(slots * 2 * kBlockM * d * sizeof(float)));
  }
  p.n_items = p.split_from + (blocks - p.split_from) * p.num_splits;
  p.div_bh = FastDiv(static_cast<uint32_t>(BH));
  p.div_qblk = FastDiv(static_cast<uint32_t>(p.n_qblk));
  p.div_splits = FastDiv(static_cast<uint32_t>(p.num_splits));
  cudaError_t err = timing_record(0, true, s);
  if (err == cudaSuccess) err = launch_fwd(p, d, s);
  if (err == cudaSuccess && p.split_from < blocks) err = launch_fwd_merge(p, o, lse, d, s);
  if (err == cudaSuccess) err = timing_record(0, false, s);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d) {
  bool empty = false;
  if (check_shape(B, H, N, d, 1.0f, &empty) != FA_OK || empty) return 0;
  const size_t rows = static_cast<size_t>(B) * H * N;
  return round_up(rows * sizeof(float)) + round_up(rows * d * sizeof(float));
}

size_t fa_bwd_deterministic_workspace_bytes(int B, int H, int N, int d) {
  bool empty = false;
  if (check_shape(B, H, N, d, 1.0f, &empty) != FA_OK || empty) return 0;
  const size_t rows = static_cast<size_t>(B) * H * N;
  // D only: dQ comes from the query-stationary kernel, accumulated in
  // tensor memory
  return round_up(rows * sizeof(float));
}

namespace {

int bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse,
             const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
             float scale, int causal, void* workspace, size_t workspace_bytes, void* stream,
             bool deterministic, bool pair = false) {
  bool empty = false;
  int rc = check_shape(B, H, N, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
      !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (pair && d != 128) return FA_ERR_UNSUPPORTED;
  const size_t need = deterministic ? fa_bwd_deterministic_workspace_bytes(B, H, N, d)
                                    : fa_bwd_workspace_bytes(B, H, N, d);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0) return FA_ERR_WORKSPACE;

  const int BH = B * H;
  const long long rows = static_cast<long long>(BH) * N;
  float* dsum = static_cast<float*>(workspace);
  // After D: the dQ accumulator, or the per-key-tile contributions.
  float* dq_buf = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                           round_up(static_cast<size_t>(rows) * sizeof(float)));
  float* dq_acc = deterministic ? nullptr : dq_buf;
  const int n_kblk = (N + kBlockN - 1) / kBlockN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  if (pair) {
    BwdPairParams pp;
    if (!encode_tile_map(&pp.tm_q, q, N, BH, d) || !encode_tile_map(&pp.tm_do, dout, N, BH, d) ||
        !encode_tile_map(&pp.tm_q64, q, N, BH, d, 64) ||
        !encode_tile_map(&pp.tm_do64, dout, N, BH, d, 64) ||
        !encode_tile_map(&pp.tm_k, k, N, BH, d) || !encode_tile_map(&pp.tm_v, v, N, BH, d))
      return FA_ERR_CUDA;
    pp.lse = lse;
    pp.dsum = dsum;
    pp.dq_acc = dq_acc;
    pp.dk = dk;
    pp.dv = dv;
    pp.status = status_ptr();
    if (!pp.status) return FA_ERR_CUDA;
    pp.N = N;
    pp.BH = BH;
    pp.n_kblk = n_kblk;
    pp.n_kpair = (n_kblk + 1) / 2;
    pp.causal = causal;
    pp.c = scale * 1.4426950408889634f;
    pp.scale = scale;
    pp.inv_scale = 1.0f / scale;
    if (2LL * pp.n_kpair * BH > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (launch_bwd_pre(o, dout, dsum, dq_acc, rows, d, s) != cudaSuccess) return FA_ERR_CUDA;
    if (timing_record(1, true, s) != cudaSuccess) return FA_ERR_CUDA;
    if (launch_bwd_pair(pp, s) != cudaSuccess) return FA_ERR_CUDA;
    if (timing_record(1, false, s) != cudaSuccess) return FA_ERR_CUDA;
    if (launch_bwd_post(dq_acc, dq, rows * d, scale, s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }

  if (deterministic) {
    // dK, dV by the key-stationary kernel without its dQ product, then dQ by
    // query-stationary CTAs that add the key tiles in order in tensor memory
    BwdParams p;
    BwdDqParams dp;
    if (!encode_tile_map(&p.tm_q, q, N, BH, d) || !encode_tile_map(&p.tm_k, k, N, BH, d) ||
        !encode_tile_map(&p.tm_v, v, N, BH, d) || !encode_tile_map(&p.tm_do, dout, N, BH, d) ||
        !encode_tile_map(&p.tm_dk, dk, N, BH, d) || !encode_tile_map(&p.tm_dv, dv, N, BH, d) ||
        !encode_tile_map(&dp.tm_dq, dq, N, BH, d))
      return FA_ERR_CUDA;
    dp.tm_q = p.tm_q;
    dp.tm_k = p.tm_k;
    dp.tm_v = p.tm_v;
    dp.tm_do = p.tm_do;
    p.tm_dq = p.tm_q;  // unused without the dQ product
    p.lse = dp.lse = lse;
    p.dsum = dp.dsum = dsum;
    p.dq_acc = nullptr;
    p.dq_part = nullptr;
    p.dk = dk;
    p.dv = dv;
    p.status = dp.status = status_ptr();
    if (!p.status) return FA_ERR_CUDA;
    p.N = dp.N = N;
    p.BH = dp.BH = BH;
    p.n_kblk = n_kblk;
    dp.n_qtiles = (N + kBlockM - 1) / kBlockM;
    p.causal = dp.causal = causal;
    p.c = dp.c = scale * 1.4426950408889634f;
    p.scale = dp.scale = scale;
    p.inv_scale = 1.0f / scale;
    p.log2e = 1.4426950408889634f;
    if (static_cast<long long>(n_kblk) * BH > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (launch_bwd_pre(o, dout, dsum, nullptr, rows, d, s) != cudaSuccess) return FA_ERR_CUDA;
    if (timing_record(1, true, s) != cudaSuccess) return FA_ERR_CUDA;
    if (launch_bwd_dkdv(p, d, s) != cudaSuccess) return FA_ERR_CUDA;
    if (launch_bwd_dq(dp, d, s) != cudaSuccess) return FA_ERR_CUDA;
    if (timing_record(1, false, s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }

  BwdParams p;
  if (!encode_tile_map(&p.tm_q, q, N, BH, d) || !encode_tile_map(&p.tm_k, k, N, BH, d) ||
      !encode_tile_map(&p.tm_v, v, N, BH, d) || !encode_tile_map(&p.tm_do, dout, N, BH, d) ||
      !encode_tile_map(&p.tm_dk, dk, N, BH, d) || !encode_tile_map(&p.tm_dv, dv, N, BH, d) ||
      !encode_dq_map(&p.tm_dq, dq_buf, N, BH, d))
    return FA_ERR_CUDA;
  p.lse = lse;
  p.dsum = dsum;
  p.dq_acc = dq_acc;
  p.dq_part = nullptr;
  p.dk = dk;
  p.dv = dv;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = N;
  p.BH = BH;
  p.n_kblk = n_kblk;
  p.causal = causal;
  p.c = scale * 1.4426950408889634f;
  p.scale = scale;
  p.inv_scale = 1.0f / scale;
  p.log2e = 1.4426950408889634f;
  if (static_cast<long long>(p.n_kblk) * BH > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;

  if (launch_bwd_pre(o, dout, dsum, dq_acc, rows, d, s) != cudaSuccess) return FA_ERR_CUDA;
  if (timing_record(1, true, s) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_bwd_main(p, d, s) != cudaSuccess) return FA_ERR_CUDA;
  if (timing_record(1, false, s) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_bwd_post(dq_acc, dq, rows * d, scale, s) != cudaSuccess) return FA_ERR_CUDA;
  return FA_OK;
}

}  // namespace

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
           const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
           float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                  workspace_bytes, stream, false);
}

int fa_bwd_2cta(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                  workspace_bytes, stream, false, true);
}

int fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                  workspace_bytes, stream, true);
}

namespace {

// Shape checks of the sliding-window calls.
int check_window(int B, int H, int Hkv, int N, int d, float scale, int window, int sinks, bool* empty) {
  if (Hkv < 0) return FA_ERR_INVALID_ARG;
  const int rc = check_shape(B, H, N, d, scale, empty);
  if (rc != FA_OK) return rc;
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (sinks > kMaxSinks) return FA_ERR_UNSUPPORTED;
  if (*empty) return FA_OK;
  if (Hkv == 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  // key positions plus a window, and the tiles of a group's heads, are ints
  if (N > (1 << 30) || static_cast<long long>(H / Hkv) * ((N + kBlockM - 1) / kBlockM) > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// How fa_window.cu cuts the queries of a key head: about two CTAs per SM
// in all (what its shared memory allows), a part of 16 rows at
// least, 256 parts at most (the join reads them all).  Nothing when no query's window leaves a first token.
struct SinkParts {
  int slots = 0, slot_rows = 0, sink_rows = 0;
  size_t bytes = 0;
};
SinkParts sink_parts(int B, int Hkv, int N, int d, int window, int sinks) {
  SinkParts s;
  if (sinks == 0 || N <= window) return s;
  const long long heads = static_cast<long long>(B) * Hkv;
  const int sms = sm_count();
  long long slots = 2 * (sms > 0 ? sms : 152) / heads;  // (without a device: a size for GB300)
  if (slots > 256) slots = 256;
  if (slots < 1) slots = 1;
  const int per = static_cast<int>((N + slots - 1) / slots);
  s.slot_rows = (per + 15) / 16 * 16;
  s.slots = (N + s.slot_rows - 1) / s.slot_rows;
  s.sink_rows = (sinks + 15) / 16 * 16;
  s.bytes = round_up(static_cast<size_t>(s.slots + 1) * heads * 2 * s.sink_rows * d * sizeof(float));
  return s;
}

// How the main kernel cuts its last round: items (key tile of a key head) run one
// per SM, in order; those of a last round that would leave SMs idle are cut into
// as many parts as fill it, a query tile each at least.  (B = 2, H = 16, Hkv = 4,
// N = 8192, d = 128, window 1024, 512 items: 392 us, unsplit 414.)
struct TileParts {
  int from = 0, parts = 1;
  size_t bytes = 0;
};
TileParts tile_parts(int B, int H, int Hkv, int N, int d, int window) {
  TileParts t;
  const int items = ((N + kBlockN - 1) / kBlockN) * B * Hkv;
  const int sms = sm_count();
  t.from = items;
  if (sms <= 0) return t;
  const int tail = items % sms;
  if (tail == 0) return t;
  const long long tiles = static_cast<long long>(H / Hkv) * ((window < N ? window : N) / kBlockM + 1);
  const int parts = static_cast<int>(sms / tail < tiles ? sms / tail : tiles);
  if (parts < 2) return t;
  t.from = items - tail;
  t.parts = parts;
  t.bytes = round_up(static_cast<size_t>(tail) * parts * 2 * kBlockN * d * sizeof(float));
  return t;
}

}  // namespace

int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv,
                  int N, int d, float scale, int window, int sinks, void* stream) {
  bool empty = false;
  const int rc = check_window(B, H, Hkv, N, d, scale, window, sinks, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse))
    return FA_ERR_INVALID_ARG;
  FwdParams p = {};
  const int BH = B * H, group = H / Hkv;
  if (!encode_tile_map(&p.tm_q, q, N, BH, d) || !encode_tile_map(&p.tm_k, k, N, B * Hkv, d) ||
      !encode_tile_map(&p.tm_v, v, N, B * Hkv, d) || !encode_tile_map(&p.tm_o, o, N, BH, d))
    return FA_ERR_CUDA;
  p.o = o;
  p.lse = lse;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = N;
  p.BH = BH;
  p.causal = 1;
  p.c = scale * 1.4426950408889634f;
  p.ln2 = 0.6931471805599453f;
  p.num_splits = 1;
  p.window = window < N ? window : N;
  p.sinks = sinks < N ? sinks : N;
  p.win_tiles = group % 2 == 0 ? 1 : 2;
  p.n_qblk = (N + p.win_tiles * kBlockM - 1) / (p.win_tiles * kBlockM);
  const int units = p.win_tiles == 1 ? BH / 2 : BH;
  if (static_cast<long long>(p.n_qblk) * units > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  p.n_items = p.n_qblk * units;
  p.split_from = p.n_items;
  p.div_bh = FastDiv(static_cast<uint32_t>(units));
  p.div_qblk = FastDiv(static_cast<uint32_t>(p.n_qblk));
  p.div_group = FastDiv(static_cast<uint32_t>(group));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err = timing_record(0, true, s);
  if (err == cudaSuccess) err = launch_fwd(p, d, s);
  if (err == cudaSuccess) err = timing_record(0, false, s);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_window_workspace_bytes(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  bool empty = false;
  if (check_window(B, H, Hkv, N, d, 1.0f, window, sinks, &empty) != FA_OK || empty) return 0;
  if (static_cast<long long>((N + kBlockN - 1) / kBlockN) * B * Hkv > 0x7fffffffLL) return 0;
  return fa_bwd_workspace_bytes(B, H, N, d) + sink_parts(B, Hkv, N, d, window, sinks).bytes +
         tile_parts(B, H, Hkv, N, d, window).bytes;
}

int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dout, void* dq, void* dk, void* dv, int B, int H, int Hkv, int N, int d,
                  float scale, int window, int sinks, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty = false;
  const int rc = check_window(B, H, Hkv, N, d, scale, window, sinks, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
      !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_INVALID_ARG;
  const int BH = B * H, BHkv = B * Hkv;
  if (static_cast<long long>((N + kBlockN - 1) / kBlockN) * BHkv > 0x7fffffffLL ||
      static_cast<long long>(BHkv) * (2 * kMaxSinks) > 0x3fffffffLL)
    return FA_ERR_UNSUPPORTED;
  const size_t need = fa_bwd_window_workspace_bytes(B, H, Hkv, N, d, window, sinks);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0) return FA_ERR_WORKSPACE;

  const long long rows = static_cast<long long>(BH) * N;
  const SinkParts sp = sink_parts(B, Hkv, N, d, window, sinks);
  char* w = static_cast<char*>(workspace);
  float* dsum = reinterpret_cast<float*>(w);
  float* dq_acc = reinterpret_cast<float*>(w + round_up(static_cast<size_t>(rows) * sizeof(float)));
  float* sink_part = reinterpret_cast<float*>(w + fa_bwd_workspace_bytes(B, H, N, d));
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  BwdParams p = {};
  if (!encode_tile_map(&p.tm_q, q, N, BH, d) || !encode_tile_map(&p.tm_k, k, N, BHkv, d) ||
      !encode_tile_map(&p.tm_v, v, N, BHkv, d) || !encode_tile_map(&p.tm_do, dout, N, BH, d) ||
      !encode_tile_map(&p.tm_dk, dk, N, BHkv, d) || !encode_tile_map(&p.tm_dv, dv, N, BHkv, d) ||
      !encode_dq_map(&p.tm_dq, dq_acc, N, BH, d))
    return FA_ERR_CUDA;
  p.lse = lse;
  p.dsum = dsum;
  p.dq_acc = dq_acc;
  p.dk = dk;
  p.dv = dv;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = N;
  p.BH = BHkv;
  p.n_kblk = (N + kBlockN - 1) / kBlockN;
  p.causal = 1;
  p.c = scale * 1.4426950408889634f;
  p.scale = scale;
  p.inv_scale = 1.0f / scale;
  p.log2e = 1.4426950408889634f;
  p.window = window < N ? window : N;
  p.group = H / Hkv;
  p.sinks = sinks < N ? sinks : N;
  p.sink_rows = sp.sink_rows;
  p.sink_main = nullptr;
  const TileParts tp = tile_parts(B, H, Hkv, N, d, window);
  p.split_from = tp.from;
  p.split_parts = tp.parts;
  p.div_kblk = FastDiv(static_cast<uint32_t>(p.n_kblk));
  p.div_parts = FastDiv(static_cast<uint32_t>(tp.parts));
  p.tile_part = sink_part + sp.bytes / sizeof(float);

  WindowParams wp = {};
  wp.tile_part = p.tile_part;
  wp.split_from = tp.from;
  wp.split_parts = tp.parts;
  wp.n_kblk = p.n_kblk;
  wp.dk = static_cast<__nv_bfloat16*>(dk);
  wp.dv = static_cast<__nv_bfloat16*>(dv);
  wp.N = N;
  wp.BHkv = BHkv;
  wp.group = p.group;
  wp.scale = scale;
  wp.dq_acc = dq_acc;
  wp.dq = static_cast<__nv_bfloat16*>(dq);
  if (sp.slots > 0) {
    wp.q = static_cast<const __nv_bfloat16*>(q);
    wp.k = static_cast<const __nv_bfloat16*>(k);
    wp.v = static_cast<const __nv_bfloat16*>(v);
    wp.o = static_cast<const __nv_bfloat16*>(o);
    wp.dout = static_cast<const __nv_bfloat16*>(dout);
    wp.lse = lse;
    wp.dsum = dsum;
    wp.sink_part = sink_part;
    wp.window = p.window;
    wp.sinks = p.sinks;
    wp.sink_rows = sp.sink_rows;
    wp.slots = sp.slots;
    wp.slot_rows = sp.slot_rows;
    wp.div_tiles = FastDiv(static_cast<uint32_t>(sp.slot_rows / 16));
    wp.div_last_tiles = FastDiv(static_cast<uint32_t>((N - (sp.slots - 1) * sp.slot_rows + 15) / 16));
    wp.status = p.status;
    wp.c = p.c;
    wp.log2e = p.log2e;
    p.sink_main = sink_part + static_cast<size_t>(sp.slots) * BHkv * 2 * sp.sink_rows * d;
    if (launch_window_pre(wp, d, s) != cudaSuccess) return FA_ERR_CUDA;
  } else if (launch_bwd_pre(o, dout, dsum, dq_acc, rows, d, s) != cudaSuccess) {
    return FA_ERR_CUDA;
  }
  if (timing_record(1, true, s) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_bwd_window(p, d, s) != cudaSuccess) return FA_ERR_CUDA;
  if (timing_record(1, false, s) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_window_post(wp, d, s) != cudaSuccess) return FA_ERR_CUDA;
  return FA_OK;
}

namespace {

// A row tensor of packed sequences: alignment, and rows of d elements that do not
// overlap.
bool rows_ok(const fa_rows* t, int rows, int heads, int d) {
  if (!t || !t->data || !aligned16(t->data)) return false;
  const long long row = rows > 1 ? t->row : 0, head = heads > 1 ? t->head : 0;
  // (TMA strides are below 2^40 bytes)
  if (row < 0 || head < 0 || row % 8 != 0 || head % 8 != 0 || row >= 1LL << 38 || head >= 1LL << 38) return false;
  if ((rows > 1 && row < d) || (heads > 1 && head < d)) return false;
  if (rows <= 1 || heads <= 1) return true;
  return row <= head ? (head - d) / row >= rows - 1 : (row - d) / head >= heads - 1;
}

// As passed to kernels, which multiply strides that may not matter by 0.
long long row_stride(const fa_rows& t, int rows) { return rows > 1 ? t.row : 0; }
long long head_stride(const fa_rows& t, int heads) { return heads > 1 ? t.head : 0; }

constexpr int kMaxPacked = 1 << 30;  // rows and sequences

// Checks shared by the calls on packed rows.  Returns FA_OK or the error; *empty:
// nothing to do.
int check_packed(const void* plan, int sequences, int rows, int H, int Hkv, int d, float scale, bool* empty) {
  *empty = false;
  if (sequences < 0 || rows < 0 || H < 0 || Hkv < 0) return FA_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (sequences > kMaxPacked || rows > kMaxPacked) return FA_ERR_UNSUPPORTED;
  if (sequences == 0 || rows == 0 || H == 0) {
    *empty = true;
    return FA_OK;
  }
  if (Hkv == 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!plan || (reinterpret_cast<uintptr_t>(plan) & (kWsAlign - 1)) != 0) return FA_ERR_INVALID_ARG;
  // work items, and a group's tiles of a sequence, are ints
  if (packed_tiles(rows, sequences, kBlockM) * H > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace

size_t fa_packed_plan_bytes(int sequences, int rows) {
  if (sequences < 0 || rows <= 0 || sequences > kMaxPacked || rows > kMaxPacked) return 0;
  return packed_layout(rows, sequences).bytes;
}

int fa_packed_plan(const int* cu_seqlens, int sequences, int rows, int causal, void* plan, size_t plan_bytes,
                   void* stream) {
  if (sequences < 0 || rows < 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (sequences > kMaxPacked || rows > kMaxPacked) return FA_ERR_UNSUPPORTED;
  if (rows == 0) return FA_OK;
  if (!cu_seqlens || !aligned4(cu_seqlens)) return FA_ERR_INVALID_ARG;
  if (!plan || plan_bytes < fa_packed_plan_bytes(sequences, rows) ||
      (reinterpret_cast<uintptr_t>(plan) & (kWsAlign - 1)) != 0)
    return FA_ERR_WORKSPACE;
  PackedPlanParams p = {};
  p.cu = cu_seqlens;
  p.sequences = sequences;
  p.rows = rows;
  p.causal = causal;
  p.plan = plan;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_packed_plan(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace {

// Key ranges that the forward may cut an item into (1: none) in a call of too few items
// for the SMs; the kernel takes as many as the lengths ask for.  The lengths are on the
// device: here their mean stands for them, empty sequences counted.  So a long sequence
// beside many short or empty ones is not cut: 16384 rows, H 1, are, with 15 sequences of
// 20 rows beside them they are not.  Whole call on the GPU, with
// and without (us; one causal sequence, d = 128): 1500 rows, H 1: 23 and 28; 2048 rows, H 2:
// 25 and 35; 8192, H 2: 52 and 106; 16384, H 1: 79 and 195.  fp32 parts and the join cost
// 5 to 10, so that from half the SMs in items on only long sequences gain (H 3, d = 128:
// 8192 rows, 99 items: 82 and 108; 4 x 2048, 108 items, not causal: 49 and 37), and under
// 1408 rows a sequence little or nothing does (3 x 1300, H 3, not causal: 35 and 29).
int packed_ranges(int sequences, int rows, int H, int Hkv) {
  const int sms = sm_count() > 0 ? sm_count() : 152;  // (without a device: a size for GB300)
  const bool pairs = H / Hkv % 2 == 0;
  const long long entries = packed_tiles(rows, sequences, pairs ? kBlockM : 2 * kBlockM);
  const long long items = entries * (pairs ? H / 2 : H);
  const int mean = rows / sequences / kBlockN;  // key tiles of a sequence
  if (mean < 11 || items > (mean < 32 ? sms / 2 : sms * 2 / 3)) return 1;
  return static_cast<int>(std::min<long long>(kMaxPackParts, 2 * sms / items + 1));
}

}  // namespace

size_t fa_fwd_packed_workspace_bytes(int sequences, int rows, int H, int Hkv, int d) {
  bool empty = false;
  // (any aligned address stands for the plan)
  if (check_packed(reinterpret_cast<const void*>(kWsAlign), sequences, rows, H, Hkv, d, 1.0f, &empty) != FA_OK || empty)
    return 0;
  const int ranges = packed_ranges(sequences, rows, H, Hkv);
  if (ranges < 2) return 0;
  const size_t n = static_cast<size_t>(ranges) * rows * H;
  return kWsAlign + round_up(n * d * sizeof(float)) + round_up(n * sizeof(float));
}

int fa_fwd_packed(const void* plan, int sequences, int rows, const fa_rows* q, const fa_rows* k, const fa_rows* v,
                  const fa_rows* o, float* lse, int H, int Hkv, int d, float scale, void* workspace,
                  size_t workspace_bytes, void* stream) {
  bool empty = false;
  const int rc = check_packed(plan, sequences, rows, H, Hkv, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!rows_ok(q, rows, H, d) || !rows_ok(k, rows, Hkv, d) || !rows_ok(v, rows, Hkv, d) || !rows_ok(o, rows, H, d) ||
      !lse || !aligned4(lse))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_fwd_packed_workspace_bytes(sequences, rows, H, Hkv, d);
  if (workspace && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0))
    return FA_ERR_WORKSPACE;
  FwdParams p = {};
  if (!encode_rows_map(&p.tm_q, *q, rows, H, d) || !encode_rows_map(&p.tm_k, *k, rows, Hkv, d) ||
      !encode_rows_map(&p.tm_v, *v, rows, Hkv, d) || !encode_rows_map(&p.tm_o, *o, rows, H, d, 32))
    return FA_ERR_CUDA;
  p.o = o->data;
  p.o_row = row_stride(*o, rows);
  p.o_head = head_stride(*o, H);
  p.lse = lse;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = rows;
  p.H = H;
  p.plan = plan;
  p.sequences = sequences;
  p.c = scale * 1.4426950408889634f;
  p.ln2 = 0.6931471805599453f;
  p.num_splits = 1;
  if (workspace && need > 0) {
    p.num_splits = packed_ranges(sequences, rows, H, Hkv);
    p.part_count = static_cast<int*>(workspace);
    p.o_part = static_cast<float*>(workspace) + kWsAlign / sizeof(float);
    p.lse_part = p.o_part + round_up(static_cast<size_t>(p.num_splits) * rows * H * d * sizeof(float)) / sizeof(float);
  }
  const int group = H / Hkv;
  p.win_tiles = group % 2 == 0 ? 1 : 2;
  const PackedLayout l = packed_layout(rows, sequences);
  p.list = reinterpret_cast<const int4*>(static_cast<const char*>(plan) + (p.win_tiles == 1 ? l.tiles : l.blocks));
  const int units = p.win_tiles == 1 ? H / 2 : H;
  // an upper bound: the kernel reads how many there are (its grid is no larger than this)
  p.n_items = static_cast<int>(packed_tiles(rows, sequences, p.win_tiles * kBlockM) * units) * p.num_splits;
  p.div_bh = FastDiv(static_cast<uint32_t>(units));
  p.div_group = FastDiv(static_cast<uint32_t>(group));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err = timing_record(0, true, s);
  if (err == cudaSuccess) err = launch_fwd(p, d, s);
  if (err == cudaSuccess && p.num_splits > 1) err = launch_packed_merge(p, d, s);
  if (err == cudaSuccess) err = timing_record(0, false, s);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace {

// How many parts the backward cuts each item (key tile of a key head) into; the
// parts' dK and dV are joined by the kernel after the main one, which costs a part
// about as much as four query tiles.  By the mean length of a sequence (lengths are
// not known here; empty ones count, and what few long ones among short ones would gain
// is missed), causal: as many parts as leave no SM idle, of two query tiles each; as fill the SMs twice, since items differ by their place, of eight; two where
// items are long and no more than two to an SM.  At d = 64 no part may be without a
// query tile (its kernel's ring): as many as a group's heads at most.
// Measured at d = 128, causal, one sequence, one part against the rule's:
//   1024 rows, H = 16, Hkv = 2     153 us -> 42 (8 parts)
//   12000 rows, H = 8, Hkv = 1    1605 us -> 578 (3)
//   4096 rows, H = 16, Hkv = 4     302 us -> 179 (2)
//   16001 rows, H = 8, Hkv = 2    1118 us -> 1048 (2)
// and beyond it, 8 sequences of 1024 rows, H = 16, Hkv = 4: 149 us, with 2 parts 175.
int packed_parts(int sequences, int rows, int H, int Hkv, int d) {
  const int sms = sm_count() > 0 ? sm_count() : 152;  // (without a device: a size for GB300)
  const int group = H / Hkv;
  const long long items = packed_tiles(rows, sequences, kBlockN) * Hkv;
  const long long tiles = (static_cast<long long>(rows) / sequences + kBlockM - 1) / kBlockM;
  const long long mean = (tiles + 1) * group / 2;  // query tiles of an item
  auto least = [](long long a, long long b) { return a < b ? a : b; };
  long long n = least(sms / items, mean / 2);
  const long long twice = least(2 * sms / items, mean / 8);
  if (twice > n) n = twice;
  if (n < 2 && items <= 2 * sms && tiles * group >= 128) n = 2;
  n = least(n, d == 64 && group < 8 ? group : 8);
  return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace

size_t fa_bwd_packed_workspace_bytes(int sequences, int rows, int H, int Hkv, int d) {
  bool empty = false;
  // (any aligned address stands for the plan)
  if (check_packed(reinterpret_cast<const void*>(kWsAlign), sequences, rows, H, Hkv, d, 1.0f, &empty) != FA_OK || empty)
    return 0;
  const size_t n = static_cast<size_t>(rows) * H;
  if (n > 0x7fffffffu) return 0;
  const int parts = packed_parts(sequences, rows, H, Hkv, d);
  return kWsAlign + 2 * round_up(n * sizeof(float)) + round_up(n * d * sizeof(float)) +
         (parts > 1 ? round_up(static_cast<size_t>(parts) * 2 * Hkv * rows * d * sizeof(float)) : 0);
}

int fa_bwd_packed(const void* plan, int sequences, int rows, const fa_rows* q, const fa_rows* k, const fa_rows* v,
                  const fa_rows* o, const float* lse, const fa_rows* dout, const fa_rows* dq, const fa_rows* dk,
                  const fa_rows* dv, int H, int Hkv, int d, float scale, void* workspace, size_t workspace_bytes,
                  void* stream) {
  bool empty = false;
  const int rc = check_packed(plan, sequences, rows, H, Hkv, d, scale, &empty);
  if (rc != FA_OK || empty) return rc;
  const size_t n = static_cast<size_t>(rows) * H;  // 32-bit row indices
  if (n > 0x7fffffffu) return FA_ERR_UNSUPPORTED;
  for (const fa_rows* t : {q, o, dout, dq})
    if (!rows_ok(t, rows, H, d)) return FA_ERR_INVALID_ARG;
  for (const fa_rows* t : {k, v, dk, dv})
    if (!rows_ok(t, rows, Hkv, d)) return FA_ERR_INVALID_ARG;
  if (!lse || !aligned4(lse)) return FA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < fa_bwd_packed_workspace_bytes(sequences, rows, H, Hkv, d) ||
      (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0)
    return FA_ERR_WORKSPACE;
  char* w = static_cast<char*>(workspace) + kWsAlign;  // behind the counter
  float* dsum = reinterpret_cast<float*>(w);
  float* lse_heads = reinterpret_cast<float*>(w + round_up(n * sizeof(float)));
  float* dq_acc = reinterpret_cast<float*>(w + 2 * round_up(n * sizeof(float)));

  BwdParams p = {};
  if (!encode_rows_map(&p.tm_q, *q, rows, H, d) || !encode_rows_map(&p.tm_k, *k, rows, Hkv, d) ||
      !encode_rows_map(&p.tm_v, *v, rows, Hkv, d) || !encode_rows_map(&p.tm_do, *dout, rows, H, d) ||
      !encode_rows_map(&p.tm_dk, *dk, rows, Hkv, d) || !encode_rows_map(&p.tm_dv, *dv, rows, Hkv, d) ||
      (d == 64 && !encode_dq_map(&p.tm_dq, dq_acc, rows, H, d)))  // (d = 128 adds dQ from registers)
    return FA_ERR_CUDA;
  p.lse = lse_heads;
  p.dsum = dsum;
  p.dq_acc = dq_acc;
  p.dk = dk->data;
  p.dv = dv->data;
  p.dk_row = row_stride(*dk, rows);
  p.dk_head = head_stride(*dk, Hkv);
  p.dv_row = row_stride(*dv, rows);
  p.dv_head = head_stride(*dv, Hkv);
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.N = rows;
  p.BH = Hkv;
  p.n_kblk = static_cast<int>(packed_tiles(rows, sequences, kBlockN));  // an upper bound
  p.c = scale * 1.4426950408889634f;
  p.scale = scale;
  p.inv_scale = 1.0f / scale;
  p.log2e = 1.4426950408889634f;
  p.group = H / Hkv;
  p.plan = plan;
  const PackedLayout l = packed_layout(rows, sequences);
  p.tiles = reinterpret_cast<const int4*>(static_cast<const char*>(plan) + l.tiles);
  p.seq_tiles = reinterpret_cast<const int4*>(static_cast<const char*>(plan) + l.seq_tiles);
  p.sequences = sequences;
  p.div_kv = FastDiv(static_cast<uint32_t>(Hkv));
  p.split_parts = packed_parts(sequences, rows, H, Hkv, d);
  p.div_parts = FastDiv(static_cast<uint32_t>(p.split_parts));
  p.counter = static_cast<unsigned int*>(workspace);
  p.tile_part = dq_acc + round_up(n * d * sizeof(float)) / sizeof(float);

  PackedBwdParams r = {};
  r.plan = plan;
  r.sequences = sequences;
  r.rows = rows;
  r.H = H;
  r.o = static_cast<const __nv_bfloat16*>(o->data);
  r.dout = static_cast<const __nv_bfloat16*>(dout->data);
  r.o_row = row_stride(*o, rows);
  r.o_head = head_stride(*o, H);
  r.do_row = row_stride(*dout, rows);
  r.do_head = head_stride(*dout, H);
  r.lse = lse;
  r.lse_heads = lse_heads;
  r.dsum = dsum;
  r.dq_acc = dq_acc;
  r.dq = static_cast<__nv_bfloat16*>(dq->data);
  r.dq_row = row_stride(*dq, rows);
  r.dq_head = head_stride(*dq, H);
  r.scale = scale;
  r.div_h = FastDiv(static_cast<uint32_t>(H));
  r.counter = p.counter;
  r.parts = p.split_parts;
  r.Hkv = Hkv;
  r.part = p.tile_part;
  r.dk = static_cast<__nv_bfloat16*>(dk->data);
  r.dv = static_cast<__nv_bfloat16*>(dv->data);
  r.dk_row = p.dk_row;
  r.dk_head = p.dk_head;
  r.dv_row = p.dv_row;
  r.dv_head = p.dv_head;
  r.div_kv = p.div_kv;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_packed_pre(r, d, s) != cudaSuccess) return FA_ERR_CUDA;
  if (timing_record(1, true, s) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_bwd_packed(p, d, s) != cudaSuccess) return FA_ERR_CUDA;
  if (timing_record(1, false, s) != cudaSuccess) return FA_ERR_CUDA;
  return launch_packed_post(r, d, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_rotate(const fa_rows* q, const fa_rows* q_out, int H, const fa_rows* k, const fa_rows* k_out, int Hkv,
              const int* positions, int rows, int d, const float* rope, int rope_len, int rot, int interleaved,
              int backward, void* stream) {
  if (rows < 0 || H < 0 || Hkv < 0 || rope_len < 0) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (backward != 0 && backward != 1)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
  if (rows == 0 || (H == 0 && Hkv == 0)) return FA_OK;
  if (rows > kMaxPacked || static_cast<long long>(H) + Hkv > (1 << 28) ||
      (static_cast<long long>(H) + Hkv) * rows > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (!positions || !aligned4(positions) || !rope || !aligned16(rope)) return FA_ERR_INVALID_ARG;
  if (H > 0 && (!rows_ok(q, rows, H, d) || !rows_ok(q_out, rows, H, d))) return FA_ERR_INVALID_ARG;
  if (Hkv > 0 && (!rows_ok(k, rows, Hkv, d) || !rows_ok(k_out, rows, Hkv, d))) return FA_ERR_INVALID_ARG;
  RotateParams p = {};
  if (H > 0) {
    p.q = static_cast<const __nv_bfloat16*>(q->data);
    p.q_out = static_cast<__nv_bfloat16*>(q_out->data);
    p.q_row = row_stride(*q, rows);
    p.q_head = head_stride(*q, H);
    p.qo_row = row_stride(*q_out, rows);
    p.qo_head = head_stride(*q_out, H);
  }
  if (Hkv > 0) {
    p.k = static_cast<const __nv_bfloat16*>(k->data);
    p.k_out = static_cast<__nv_bfloat16*>(k_out->data);
    p.k_row = row_stride(*k, rows);
    p.k_head = head_stride(*k, Hkv);
    p.ko_row = row_stride(*k_out, rows);
    p.ko_head = head_stride(*k_out, Hkv);
  }
  p.H = H;
  p.Hkv = Hkv;
  p.positions = positions;
  p.rows = rows;
  p.rope = rope;
  p.rope_len = rope_len;
  p.rot = rot;
  p.interleaved = interleaved;
  p.backward = backward;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_rotate(p, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_block_bytes(int format, int page_size, int d) {
  if (format != FA_CACHE_BF16 && format != FA_CACHE_FP4) return 0;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return 0;
  if (d != 64 && d != 128) return 0;
  return 2 * paged_half_bytes(format == FA_CACHE_FP4, page_size, d);
}

namespace {

// A row tensor of `heads` heads: its pointer and strides.
bool row_strides_ok(const void* p, long long row, long long head, int d) {
  return p && aligned16(p) && row >= 0 && head >= 0 && row % 8 == 0 && head % 8 == 0 &&
         (head >= d || head == 0);
}

// Checks a cache descriptor and the ragged batch's tables.  Returns FA_OK or
// the error; *empty: nothing to do.
int check_cache(const fa_paged_cache* c, const int* cu_new, int rows, PagedView* view, bool* empty) {
  *empty = false;
  if (!c || c->B < 0 || c->Hkv < 0 || rows < 0 || c->num_pages < 0 || c->max_pages < 0)
    return FA_ERR_INVALID_ARG;
  if (fa_paged_block_bytes(c->format, c->page_size, c->d) == 0) return FA_ERR_UNSUPPORTED;
  if (c->B == 0 || c->Hkv == 0 || rows == 0) {
    *empty = true;
    return FA_OK;
  }
  if (c->num_pages == 0 || c->max_pages == 0) return FA_ERR_INVALID_ARG;
  if (!c->pages || !c->page_table || !c->seq_lens || !cu_new) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->pages) || !aligned4(c->page_table) || !aligned4(c->seq_lens) ||
      !aligned4(cu_new) || !aligned4(c->k_scale) || !aligned4(c->v_scale))
    return FA_ERR_INVALID_ARG;
  if (c->format != FA_CACHE_FP4 && (c->k_scale || c->v_scale)) return FA_ERR_INVALID_ARG;
  // block indices (times 2, K and V) and positions are ints in the kernels
  if (2LL * c->num_pages * c->Hkv > 0x7fffffffLL ||
      static_cast<long long>(c->max_pages) * c->page_size > 0x7fffff00LL)
    return FA_ERR_UNSUPPORTED;
  view->pages = static_cast<uint8_t*>(c->pages);
  view->page_table = c->page_table;
  view->seq_lens = c->seq_lens;
  view->k_scale = c->k_scale;
  view->v_scale = c->v_scale;
  view->B = c->B;
  view->Hkv = c->Hkv;
  view->num_pages = c->num_pages;
  view->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  view->max_pages = c->max_pages;
  return FA_OK;
}

}  // namespace

int fa_paged_append(const fa_paged_cache* cache, const void* k, long long k_row, long long k_head,
                    const void* v, long long v_row, long long v_head, const int* cu_new, int rows,
                    const void* q, long long q_row, long long q_head, void* q_out, int H,
                    const float* rope, int rope_len, int rot, int interleaved, void* stream) {
  PagedAppendParams p = {};
  bool empty = false;
  const int rc = check_cache(cache, cu_new, rows, &p.c, &empty);
  if (rc != FA_OK) return rc;
  const int d = cache->d;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || rot % 16 != 0 || rope_len < 0) return FA_ERR_INVALID_ARG;
  if (q && H < 1) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (!row_strides_ok(k, k_row, k_head, d) || !row_strides_ok(v, v_row, v_head, d))
    return FA_ERR_INVALID_ARG;
  if (q && (!row_strides_ok(q, q_row, q_head, d) || !q_out || !aligned16(q_out)))
    return FA_ERR_INVALID_ARG;
  if (rot > 0 && (!rope || !aligned16(rope))) return FA_ERR_INVALID_ARG;
  if ((q ? H : 0) + 2LL * cache->Hkv > (1 << 28)) return FA_ERR_UNSUPPORTED;  // rows of a block's tokens are an int
  p.cu = cu_new;
  p.rows = rows;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_row = k_row;
  p.k_head = k_head;
  p.v_row = v_row;
  p.v_head = v_head;
  p.q_row = q_row;
  p.q_head = q_head;
  p.H = q ? H : 0;
  p.div_q = FastDiv(static_cast<uint32_t>(q ? H : 1));
  p.div_kv = FastDiv(static_cast<uint32_t>(2 * cache->Hkv));
  p.rope = rope;
  p.rope_len = rope_len;
  p.rot = rot;
  p.interleaved = interleaved;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_paged_append(p, d, cache->format == FA_CACHE_FP4, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_paged_read(const fa_paged_cache* cache, const int* cu_new, int rows, void* k, void* v,
                  void* stream) {
  PagedReadParams p = {};
  bool empty = false;
  const int rc = check_cache(cache, cu_new, rows, &p.c, &empty);
  if (rc != FA_OK || empty) return rc;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
  p.cu = cu_new;
  p.rows = rows;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  if (2LL * cache->Hkv > (1 << 28)) return FA_ERR_UNSUPPORTED;
  p.div_heads = FastDiv(static_cast<uint32_t>(2 * cache->Hkv));
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_paged_read(p, cache->d, cache->format == FA_CACHE_FP4,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// Partial rows of every worker (two slots of a block's rows each: O, references
// and sums) and the segments' continuations.
size_t fa_fwd_paged_workspace_bytes(int d) {
  if (d != 64 && d != 128) return 0;
  const size_t slots = 2 * static_cast<size_t>(fwd_paged_workers());
  return round_up(slots * kPagedRows * d * sizeof(float)) + round_up(slots * 2 * kPagedRows * sizeof(float)) +
         round_up(slots / 2 * sizeof(int4));
}

int fa_fwd_paged(const fa_paged_cache* cache, const void* q, long long q_row, long long q_head,
                 void* o, float* lse, const int* cu_new, int rows, int max_new, int H, float scale,
                 int window, int sinks, void* workspace, size_t workspace_bytes, void* stream) {
  FwdPagedParams p = {};
  bool empty = false;
  const int rc = check_cache(cache, cu_new, rows, &p.c, &empty);
  if (rc != FA_OK) return rc;
  if (!(isfinite(scale) && scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (H < 0 || window < 0 || sinks < 0 || max_new < 0) return FA_ERR_INVALID_ARG;
  if (empty || H == 0) return FA_OK;
  if (H % cache->Hkv != 0 || max_new < 1) return FA_ERR_INVALID_ARG;
  const int d = cache->d;
  const bool fp4 = cache->format == FA_CACHE_FP4;
  if (!row_strides_ok(q, q_row, q_head, d) || !o || !lse || !aligned16(o) || !aligned4(lse))
    return FA_ERR_INVALID_ARG;
  const int group = H / cache->Hkv;
  if (static_cast<long long>(max_new) * group > 0x7fffff00LL) return FA_ERR_UNSUPPORTED;
  const long long blocks = (static_cast<long long>(max_new) * group + 15) / 16;
  if (blocks * cache->Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_fwd_paged_workspace_bytes(d);
  if (!workspace || workspace_bytes < need ||
      (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0)
    return FA_ERR_WORKSPACE;
  if (need == 0) return FA_ERR_CUDA;
  const size_t slots = 2 * static_cast<size_t>(fwd_paged_workers());
  char* w = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(w);
  w += round_up(slots * kPagedRows * d * sizeof(float));
  p.part_ml = reinterpret_cast<float*>(w);
  w += round_up(slots * 2 * kPagedRows * sizeof(float));
  p.info = reinterpret_cast<int4*>(w);
  if (!fp4) {
    if (!encode_tile_map(&p.tm, cache->pages, cache->page_size, cache->num_pages * cache->Hkv * 2, d, 16))
      return FA_ERR_CUDA;
  }
  p.cu = cu_new;
  p.rows = rows;
  p.max_new = max_new;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_row = q_row;
  p.q_head = q_head;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.H = H;
  p.group = group;
  p.window = window == 0 ? 0x7fffffff : window;
  p.sinks = sinks;
  p.scale = scale * 1.4426950408889634f;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  const long long tiles = (static_cast<long long>(cache->max_pages) * cache->page_size + 15) / 16 + 1;
  // an upper bound of the units of work, as far as it matters (the grid)
  const long long cap = 1LL << 20;
  long long units = blocks < cap ? blocks * cache->Hkv : cap;
  units = units < cap ? units * tiles : cap;
  units = units < cap ? units * cache->B : cap;
  return launch_fwd_paged(p, d, fp4, units, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_last_device_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  unsigned int word = 0;
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(&word, g_status_word, sizeof(word)) != cudaSuccess) return FA_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(zero)) != cudaSuccess) return FA_ERR_CUDA;
  g_last_site = static_cast<int>((word >> 8) & 0xFFFFu);
  const int code = static_cast<int>(word & 0xFFu);
  return code == 0 ? FA_OK : code;
}

int fa_last_device_site(void) { return g_last_site; }

int fa_timing_enable(int enable) {
  std::lock_guard<std::mutex> lock(g_timing.mu);
  g_timing.enabled = enable != 0;
  return FA_OK;
}

int fa_timing_last_ms(int kernel, float* ms) {
  if (kernel < 0 || kernel > 1 || !ms) return FA_ERR_INVALID_ARG;
  cudaEvent_t start, stop;
  {
    std::lock_guard<std::mutex> lock(g_timing.mu);
    if (!g_timing.recorded[kernel]) return FA_ERR_INVALID_ARG;
    start = g_timing.start[kernel];
    stop = g_timing.stop[kernel];
  }
  if (cudaEventSynchronize(stop) != cudaSuccess) return FA_ERR_CUDA;
  return cudaEventElapsedTime(ms, start, stop) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

unsigned long long fa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int fa_exp2_poly_eval(const float* x, float* y, long long n, void* stream) {
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!x || !y || !aligned4(x) || !aligned4(y)) return FA_ERR_INVALID_ARG;
  const long long blocks = (n + 255) / 256;
  exp2_poly_eval_kernel<<<static_cast<unsigned int>(blocks < 4096 ? blocks : 4096), 256, 0,
                          static_cast<cudaStream_t>(stream)>>>(x, y, n);
  return launched(1) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_debug_bounded_wait(unsigned long long limit_ns, void* stream) {
  if (limit_ns < 1000000ull || limit_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
  unsigned int* status = status_ptr();
  if (!status) return FA_ERR_CUDA;
  bounded_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(status, limit_ns);
  return launched(1) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
