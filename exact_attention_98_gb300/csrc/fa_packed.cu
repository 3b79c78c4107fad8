// Plans of packed sequences (fa_packed.cuh).
//
// A list is a counting sort of its tiles by cost, the key tiles that a tile
// sees: costs below 64 have a bucket each, higher ones 32 to the octave (a
// CTA's share of the work then differs by 3% at most from an exact order's).  A
// warp takes one bucket of one list: its first walk over the sequences counts the tiles of
// higher buckets, which gives the bucket's place without a word between warps,
// its second writes the bucket's tiles, in the order of the sequences, so the plan's bits do
// not vary.  Two further walks' worth of blocks write the rows' positions.
//
// Latency bounds it (cu is read from cache by every warp): 3 sequences of 300 rows
// and 24 of 24001 take about the time of a launch; it is made once for a batch.
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
      for (int t = 0; t < n; ++t) list[place + t] = make_int4(start, len, first + t, place);
    for (unsigned int left = __ballot_sync(0xffffffffu, n > 8); left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const int s = __shfl_sync(0xffffffffu, start, src), ln = __shfl_sync(0xffffffffu, len, src);
      const int f = __shfl_sync(0xffffffffu, first, src), m = __shfl_sync(0xffffffffu, n, src);
      const int pl = __shfl_sync(0xffffffffu, place, src);
      for (int t = lane; t < m; t += 32) list[pl + t] = make_int4(s, ln, f + t, pl);
    }
    at += __shfl_sync(0xffffffffu, sum, 31);
  }
}

}  // namespace

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
