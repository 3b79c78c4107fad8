// Plans of packed sequences (fa_packed.cuh).
//
// A list is a counting sort of its tiles by cost, the key tiles that a tile
// sees: costs below 64 have a bucket each, higher ones 32 to the octave (a
// CTA's share of the work then differs by 3% at most from an exact order's).  A
// warp takes one bucket of one list: its first walk over the sequences counts the tiles of
// higher buckets, which gives the bucket's place without a word between warps,
// its second writes the bucket's tiles, in the order of the sequences, so the plan's
// bits do not vary.  Further blocks write the rows' positions.
//
// Latency bounds it (cu is read from cache by every warp): 3 sequences of 300 rows
// and 24 of 24001 take 3 to 4 us; it is made once for a batch.
#include "fa_packed.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kFineCosts = 64;  // costs below it have buckets of their own

__host__ __device__ inline int cost_bucket(int cost) {
  if (cost < kFineCosts) return cost;
  int k = 6;
  while ((cost >> k) > 1) ++k;
  return kFineCosts + (k - 6) * 32 + ((cost >> (k - 5)) & 31);
}
// Costs of bucket b: [lo, hi)
__device__ __forceinline__ void bucket_costs(int b, int& lo, int& hi) {
  if (b < kFineCosts) {
    lo = b;
    hi = b + 1;
    return;
  }
  const int k = (b - kFineCosts) / 32 + 6, sub = (b - kFineCosts) % 32;
  lo = (32 + sub) << (k - 5);
  hi = (33 + sub) << (k - 5);
}

// Tiles of a sequence of nt in bucket [lo, hi): the first, and how many.
__device__ __forceinline__ int bucket_tiles(int nt, bool by_tile, int lo, int hi, int& first) {
  if (by_tile) {  // tile t costs t + 1
    first = lo - 1;
    return max(0, min(nt, hi - 1) - first);
  }
  first = 0;
  return nt >= lo && nt < hi ? nt : 0;
}
__device__ __forceinline__ int higher_tiles(int nt, bool by_tile, int hi) {
  return by_tile ? max(0, nt - (hi - 1)) : nt >= hi ? nt : 0;
}

__device__ __forceinline__ bool bad_offsets(const int* cu, int b, int rows) {
  return cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > rows;
}

__global__ void __launch_bounds__(kPlanThreads) fa_packed_plan_kernel(const __grid_constant__ PackedPlanParams p) {
  grid_dependency_wait();
  uint8_t* plan = static_cast<uint8_t*>(p.plan);
  const PackedLayout l = packed_layout(p.rows, p.sequences);
  const int lane = lane_id();
  if (static_cast<int>(blockIdx.x) >= 3 * p.list_blocks) {
    // positions: -1 where a row belongs to no sequence
    int* pos = reinterpret_cast<int*>(plan + l.positions);
    bool bad = false;
    for (int b = threadIdx.x; b < p.sequences; b += kPlanThreads) bad |= bad_offsets(p.cu, b, p.rows);
    bad = __syncthreads_or(bad);
    const int blocks = static_cast<int>(gridDim.x) - 3 * p.list_blocks;
    for (long long r = (blockIdx.x - 3LL * p.list_blocks) * kPlanThreads + threadIdx.x; r < p.rows;
         r += static_cast<long long>(blocks) * kPlanThreads) {
      int at = -1;
      if (!bad) {
        int lo = 0, hi = p.sequences;  // first b with cu[b+1] > r
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (p.cu[mid + 1] > r) hi = mid;
          else lo = mid + 1;
        }
        if (lo < p.sequences && p.cu[lo] <= r) at = static_cast<int>(r) - p.cu[lo];
      }
      pos[r] = at;
    }
    return;
  }
  const int which = static_cast<int>(blockIdx.x) / p.list_blocks;  // tiles, blocks, seq_tiles
  // heaviest bucket first; bucket 0 (no cost) has none
  const int bucket = p.buckets - 1 - ((static_cast<int>(blockIdx.x) % p.list_blocks) * kPlanWarps + warp_id());
  if (bucket < 1) return;
  const int size = which == 1 ? 2 * kBlockM : kBlockM;
  const bool by_tile = which != 2 && p.causal;
  int4* list = reinterpret_cast<int4*>(plan + (which == 0 ? l.tiles : which == 1 ? l.blocks : l.seq_tiles));
  int lo, hi;
  bucket_costs(bucket, lo, hi);
  bool bad = false;
  int total = 0, at = 0;
  for (int b = lane; b < p.sequences; b += 32) {
    bad |= bad_offsets(p.cu, b, p.rows);
    const int len = p.cu[b + 1] - p.cu[b];
    const int nt = len / size + (len % size != 0);
    total += nt;
    at += higher_tiles(nt, by_tile, hi);
  }
  bad = __any_sync(0xffffffffu, bad);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    at += __shfl_xor_sync(0xffffffffu, at, off);
  }
  if (bucket == 1 && lane == 0) {
    PackedHead* h = reinterpret_cast<PackedHead*>(plan);
    if (which == 0) {
      if (bad) record_status(p.status, kPackedInvalid, kSitePackedOffsets);
      h->magic = kPackedMagic;
      h->rows = p.rows;
      h->sequences = p.sequences;
      h->causal = p.causal;
      h->n_tiles = bad ? 0 : total;
      h->begin = bad || p.sequences == 0 ? 0 : p.cu[0];
      h->end = bad || p.sequences == 0 ? 0 : p.cu[p.sequences];
    } else if (which == 1) {
      h->n_blocks = bad ? 0 : total;
    }
  }
  if (bad) return;
  for (int b0 = 0; b0 < p.sequences; b0 += 32) {
    const int b = b0 + lane;
    int start = 0, len = 0, first = 0, n = 0;
    if (b < p.sequences) {
      start = p.cu[b];
      len = p.cu[b + 1] - start;
      n = bucket_tiles(len / size + (len % size != 0), by_tile, lo, hi, first);
    }
    int sum = n;  // of this lane and those below
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    // a lane's own tiles where there are few, all lanes together on a long sequence's
    const int place = at + sum - n;
    if (n > 0 && n <= 8)
      for (int t = 0; t < n; ++t) list[place + t] = make_int4(start, len, first + t, 0);
    for (unsigned int left = __ballot_sync(0xffffffffu, n > 8); left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const int s = __shfl_sync(0xffffffffu, start, src), ln = __shfl_sync(0xffffffffu, len, src);
      const int f = __shfl_sync(0xffffffffu, first, src), m = __shfl_sync(0xffffffffu, n, src);
      const int pl = __shfl_sync(0xffffffffu, place, src);
      for (int t = lane; t < m; t += 32) list[pl + t] = make_int4(s, ln, f + t, 0);
    }
    at += __shfl_sync(0xffffffffu, sum, 31);
  }
}

// Before the backward's main kernel: D = rowsum(dO * O) and LSE by heads, where the
// main kernel reads a head's rows one after another, and the zeroed dQ
// accumulator.  16 bytes of a row to a lane.  Rows of no sequence are left out.
// After it: dQ = scale * accumulator -> bf16, and dK and dV from their parts, where the
// main kernel's items are split, in order.  Both are bound by HBM: 16384 rows, H = 16,
// d = 128: 38 us for 268 MB (7.1 TB/s) and 26.5 for 201 MB (part of them still in L2).
constexpr int kRowThreads = 256;

template <int D>
__global__ void __launch_bounds__(kRowThreads) fa_packed_pre_kernel(const __grid_constant__ PackedBwdParams p) {
  constexpr int kLanes = D / 8;
  grid_dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0u;
  const PackedHead& head = *static_cast<const PackedHead*>(p.plan);
  if (!packed_fits(head, p.rows, p.sequences)) return;  // (the main kernel records it)
  const int col = static_cast<int>(threadIdx.x) % kLanes * 8;
  const long long n = static_cast<long long>(head.end - head.begin) * p.H;
  // (whole warps leave the loop together: a warp's rows are neighbours)
  for (long long i0 = blockIdx.x * static_cast<long long>(kRowThreads / kLanes); i0 < n;
       i0 += static_cast<long long>(gridDim.x) * (kRowThreads / kLanes)) {
    const long long i = i0 + threadIdx.x / kLanes;
    float acc = 0.0f;
    size_t at = 0;
    long long row = 0;
    int h = 0;
    if (i < n) {
      const uint32_t t = p.div_h.div(static_cast<uint32_t>(i));
      row = head.begin + static_cast<long long>(t);
      h = static_cast<int>(static_cast<uint32_t>(i) - t * p.div_h.d);
      at = static_cast<size_t>(h) * p.rows + row;
      const uint4 a = *reinterpret_cast<const uint4*>(p.o + row * p.o_row + h * p.o_head + col);
      const uint4 b = *reinterpret_cast<const uint4*>(p.dout + row * p.do_row + h * p.do_head + col);
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
      const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 x = __bfloat1622float2(a2[c]), y = __bfloat1622float2(b2[c]);
        acc = fmaf(x.x, y.x, acc);
        acc = fmaf(x.y, y.y, acc);
      }
      float4* z = reinterpret_cast<float4*>(p.dq_acc + at * D + col);
      z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (i < n && col == 0) {
      p.dsum[at] = acc;
      p.lse_heads[at] = p.lse[row * p.H + h];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) fa_packed_post_kernel(const __grid_constant__ PackedBwdParams p) {
  constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes, kUnroll = 4;
  grid_dependency_wait();
  const PackedHead& head = *static_cast<const PackedHead*>(p.plan);
  if (!packed_fits(head, p.rows, p.sequences)) return;
  const int col = static_cast<int>(threadIdx.x) % kLanes * 8;
  const long long n = static_cast<long long>(head.end - head.begin) * p.H;
  for (long long i0 = blockIdx.x * static_cast<long long>(kRows * kUnroll) + threadIdx.x / kLanes; i0 < n;
       i0 += static_cast<long long>(gridDim.x) * (kRows * kUnroll)) {
    float4 a[kUnroll], b[kUnroll];
    __nv_bfloat16* to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = i0 + u * kRows;
      to[u] = nullptr;
      if (i < n) {
        const uint32_t t = p.div_h.div(static_cast<uint32_t>(i));
        const long long row = head.begin + static_cast<long long>(t);
        const int h = static_cast<int>(static_cast<uint32_t>(i) - t * p.div_h.d);
        const float4* from = reinterpret_cast<const float4*>(p.dq_acc + (static_cast<size_t>(h) * p.rows + row) * D + col);
        a[u] = from[0];
        b[u] = from[1];
        to[u] = p.dq + row * p.dq_row + h * p.dq_head + col;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (to[u] != nullptr)
        *reinterpret_cast<uint4*>(to[u]) =
            make_uint4(pack_bf16x2(a[u].x * p.scale, a[u].y * p.scale), pack_bf16x2(a[u].z * p.scale, a[u].w * p.scale),
                       pack_bf16x2(b[u].x * p.scale, b[u].y * p.scale), pack_bf16x2(b[u].z * p.scale, b[u].w * p.scale));
  }
  if (p.parts < 2) return;
  const long long m = 2LL * (head.end - head.begin) * p.Hkv;
  const size_t stride = 2 * static_cast<size_t>(p.Hkv) * p.rows * D;  // of a part
  for (long long i = blockIdx.x * static_cast<long long>(kRows) + threadIdx.x / kLanes; i < m;
       i += static_cast<long long>(gridDim.x) * kRows) {
    const int dv = static_cast<int>(i & 1);
    const uint32_t th = static_cast<uint32_t>(i >> 1), t = p.div_kv.div(th);
    const long long row = head.begin + static_cast<long long>(t);
    const int h = static_cast<int>(th - t * p.div_kv.d);
    const float* from = p.part + ((static_cast<size_t>(dv) * p.Hkv + h) * p.rows + row) * D + col;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
    for (int k = 0; k < p.parts; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(from + k * stride);
      const float4 y = *reinterpret_cast<const float4*>(from + k * stride + 4);
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
    const float mul = dv ? 1.0f : p.scale;
    __nv_bfloat16* to = dv ? p.dv + row * p.dv_row + h * p.dv_head : p.dk + row * p.dk_row + h * p.dk_head;
    *reinterpret_cast<uint4*>(to + col) =
        make_uint4(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul),
                   pack_bf16x2(b.x * mul, b.y * mul), pack_bf16x2(b.z * mul, b.w * mul));
  }
}

// The forward's parts joined: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
// Parts without a key have LSE_s = -inf and are not read.  In fp32, rounded once, at the end.
// Bound by latency: the parts, at most some 60 MB, come from L2.
template <int D>
__global__ void __launch_bounds__(kRowThreads) fa_packed_merge_kernel(const __grid_constant__ FwdParams p) {
  constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes;
  grid_dependency_wait();
  const PackedHead& head = *static_cast<const PackedHead*>(p.plan);
  if (!packed_fits(head, p.N, p.sequences)) return;
  const int parts = *p.part_count;
  const int col = static_cast<int>(threadIdx.x) % kLanes * 8;
  const long long n = static_cast<long long>(head.end - head.begin) * p.H;
  const size_t stride = static_cast<size_t>(p.N) * p.H;  // of a part
  for (long long i = blockIdx.x * static_cast<long long>(kRows) + threadIdx.x / kLanes; i < n;
       i += static_cast<long long>(gridDim.x) * kRows) {
    const size_t at = static_cast<size_t>(head.begin) * p.H + i;  // row * H + head
    // four ranges at a time: their loads together
    float m = -INFINITY;
    for (int s0 = 0; s0 < parts; s0 += 4) {
      float ls[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) ls[u] = s0 + u < parts ? p.lse_part[(s0 + u) * stride + at] : -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) m = fmaxf(m, ls[u]);
    }
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.0f;
    for (int s0 = 0; s0 < parts; s0 += 4) {
      float w[4];
      float4 x[4], y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float ls = s0 + u < parts ? p.lse_part[(s0 + u) * stride + at] : -INFINITY;
        w[u] = 0.0f;
        x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ls != -INFINITY) {
          w[u] = expf(ls - m);
          const float4* from = reinterpret_cast<const float4*>(p.o_part + ((s0 + u) * stride + at) * D + col);
          x[u] = from[0];
          y[u] = from[1];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        sum += w[u];
        acc[0] += w[u] * x[u].x; acc[1] += w[u] * x[u].y; acc[2] += w[u] * x[u].z; acc[3] += w[u] * x[u].w;
        acc[4] += w[u] * y[u].x; acc[5] += w[u] * y[u].y; acc[6] += w[u] * y[u].z; acc[7] += w[u] * y[u].w;
      }
    }
    const float inv = 1.0f / sum;
    const long long row = head.begin + i / p.H;
    const int h = static_cast<int>(i % p.H);
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.o) + row * p.o_row + h * p.o_head + col;
    *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                                               pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (col == 0) p.lse[at] = m + logf(sum);
  }
}

// Blocks for n rows of a head: as many as are resident at once, at most.
dim3 row_grid(long long n, int per_block) {
  const long long blocks = (n + per_block - 1) / per_block, cap = 8LL * (sm_count() > 0 ? sm_count() : 1);
  return dim3(static_cast<unsigned int>(blocks < cap ? blocks : cap));
}

}  // namespace

cudaError_t launch_packed_pre(const PackedBwdParams& p, int d, cudaStream_t stream) {
  const cudaError_t err = launch_dependent(d == 128 ? fa_packed_pre_kernel<128> : fa_packed_pre_kernel<64>,
                                           row_grid(static_cast<long long>(p.rows) * p.H, kRowThreads / (d / 8)),
                                           dim3(kRowThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_packed_post(const PackedBwdParams& p, int d, cudaStream_t stream) {
  const cudaError_t err = launch_dependent(d == 128 ? fa_packed_post_kernel<128> : fa_packed_post_kernel<64>,
                                           row_grid(static_cast<long long>(p.rows) * p.H, 4 * kRowThreads / (d / 8)),
                                           dim3(kRowThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_packed_merge(const FwdParams& p, int d, cudaStream_t stream) {
  const cudaError_t err = launch_dependent(d == 128 ? fa_packed_merge_kernel<128> : fa_packed_merge_kernel<64>,
                                           row_grid(static_cast<long long>(p.N) * p.H, kRowThreads / (d / 8)),
                                           dim3(kRowThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_packed_plan(PackedPlanParams p, cudaStream_t stream) {
  // the last bucket that a sequence of all the rows reaches
  p.buckets = cost_bucket((p.rows + kBlockM - 1) / kBlockM) + 1;
  p.list_blocks = (p.buckets - 1 + kPlanWarps - 1) / kPlanWarps;
  const int row_blocks = (p.rows + kPlanThreads - 1) / kPlanThreads;
  const int cap = 8 * (sm_count() > 0 ? sm_count() : 1);
  const cudaError_t err =
      launch_dependent(fa_packed_plan_kernel, dim3(3 * p.list_blocks + (row_blocks < cap ? row_blocks : cap)),
                       dim3(kPlanThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

}  // namespace fa
