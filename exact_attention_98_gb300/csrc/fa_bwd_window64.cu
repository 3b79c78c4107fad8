// Backward of the sliding window with shared key heads at d = 64 (d = 128 runs
// fa_bwd.cu's body): the key-stationary products of fa_bwd.cu (S^T = K Q_i^T,
// dP^T = V dO_i^T, dV += P^T dO_i, dK += dS^T Q_i, dQ_i = dS K, all tcgen05 into
// tensor memory, same columns and operand layouts), over the query tiles whose
// windows reach the key tile, of each query head of the group in turn: dV and dK
// of a shared key head accumulate in tensor memory over the whole group.
//
// An item is a key tile of a key head.  A short window leaves it few query
// tiles (window / 128 + 1 per head) of little work each at d = 64, so what a CTA
// does once per item weighs: the CTAs are persistent, and every role walks on
// into the next item on its own.  K and V have two buffers, so that the next item's
// first products follow this one's last as any tile's do; dV and dK are written
// out beside them (a barrier, kBarAccFree, keeps its first dV from the accumulator
// until they have left it).  Barriers and tensor memory are set up once.
//
// Order of a tile's products: dV_i, S^T_{i+1}, dK_i, dP^T_{i+1}, dQ_i, each once
// the compute warps have left its operand: the next tile's S^T and dP^T are not
// behind dQ_i, whose dS goes through shared memory.
//
// Masks: key j sees the queries j <= i < j + window, which cuts the diagonal
// tile and the last one or two of a head.  (First tokens' pairs outside the
// window are fa_window.cu's.)
//
// Code size: the roles' loops run side by side, and a tile takes a few thousand
// cycles, so instruction fetch is what a long body pays with.  Therefore one copy
// of each product's issue, waits in few instructions, a mask after the one copy of
// the exponentials, and 32-bit item arithmetic with precomputed divisors: 106 KB
// of code were 92 us, 68 KB are 67.6 (B = 2, H = Hkv = 16, N = 4096, window 512).
//
// What bounds it (same sizes; 67.6 us, 0.6 PFLOP/s of the five products): the
// chain of a tile, about 2900 cycles: exponentials (1100, the MUFU's rate), dV and
// the next S^T behind them (900), commit and wake-up; dS and its way through shared
// memory fit beside.  An item's change costs another 3000.
//
// dS is formed from P as computed, not as rounded to bf16 for the dV product:
// that rounding would add to dQ and dK as much as dS's own.
#include "fa_device.cuh"
#include "fa_kernels.h"

namespace fa {
namespace {

constexpr int D = 64;

struct WinCfg {
  static constexpr int kThreads = 512;
  static constexpr int kLaunchRegs = 128;
  static constexpr int kComputeRegs = 144;  // 2 x 128 threads
  static constexpr int kDrainRegs = 144;    // 128 threads: a dQ row in registers
  static constexpr int kOtherRegs = 80;     // 128 threads (load, MMA)
  static_assert(2 * 128 * kComputeRegs + 128 * kDrainRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
                "register split exceeds the launch allocation");
  static constexpr int kComputeWarps = 8;
  static constexpr int kDrainWarp0 = 8;
  static constexpr int kProducerWarp = 12;
  static constexpr int kMmaWarp = 13;
  static constexpr int kKVWarp = 14;  // loads K and V (the producer runs tiles ahead of them)
  static constexpr int kTileBytes = kBlockM * D * 2;
  static constexpr int kHalfBytes = kBlockM * 64 * 2;
  static constexpr int kStages = 3;
  static constexpr int kKOff = 0;  // two buffers each
  static constexpr int kVOff = 2 * kTileBytes;
  static constexpr int kQOff = 4 * kTileBytes;
  static constexpr int kDOOff = kQOff + kStages * kTileBytes;
  // per stage the fp32 rows -LSE log2 e and -D, which the compute warps apply
  static constexpr int kRowsOff = kDOOff + kStages * kTileBytes;
  static constexpr int kRowBytes = kBlockM * 4;
  static constexpr int kDsOff = kRowsOff + kStages * 2 * kRowBytes;
  static constexpr int kDsBytes = kBlockN * kBlockM * 2;
  static constexpr int kDqCols = 16;
  static constexpr int kDqChunks = D / kDqCols;
  static constexpr int kDqChunkBytes = kBlockM * kDqCols * 4;
  static constexpr int kDqBufs = 3;
  static constexpr int kDqOff = kDsOff + kDsBytes;
  static constexpr int kBarOff = kDqOff + kDqBufs * kDqChunkBytes;
  static constexpr int kBarKV = 0;  // K and V in buffer m % 2
  static constexpr int kBarStFull = 2;
  static constexpr int kBarStEmpty = kBarStFull + kStages;
  static constexpr int kBarSFull = kBarStEmpty + kStages;
  static constexpr int kBarDPFull = kBarSFull + 1;
  static constexpr int kBarPFull = kBarDPFull + 1;
  static constexpr int kBarDSTmem = kBarPFull + 1;
  static constexpr int kBarDSFull = kBarDSTmem + 1;
  static constexpr int kBarDQFull = kBarDSFull + 1;
  static constexpr int kBarDQEmpty = kBarDQFull + 1;
  static constexpr int kBarMmaDone = kBarDQEmpty + 1;  // an item's products are complete
  static constexpr int kBarAccFree = kBarMmaDone + 1;  // its dV and dK have left tensor memory
  static constexpr int kBarKVFree = kBarAccFree + 1;   // its dV and dK have left K's and V's buffer
  static constexpr int kNumBars = kBarKVFree + 1;
  static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  static constexpr int kSmemBytes = kAbortOff + 4 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;
  static constexpr uint32_t kColDP = 128;
  static constexpr uint32_t kColDV = 256;
  static constexpr uint32_t kColDK = 256 + D;
  static constexpr uint32_t kColDQ = 256 + 2 * D;
  static_assert(kColDQ + D <= 512, "tensor-memory columns");
  static constexpr int kDrainBarrier = 1;
  static constexpr int kEpiBarrier0 = 2;  // and 3: one per compute warpgroup
  static __device__ __forceinline__ uint32_t packed_col(int kk) {
    return static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8);
  }
};

enum : unsigned int {
  kSiteKV = 0x211,
  kSiteStFull = 0x212,
  kSiteStEmpty = 0x213,
  kSiteSFull = 0x214,
  kSiteDPFull = 0x215,
  kSitePFull = 0x216,
  kSiteDSFull = 0x218,
  kSiteDQFull = 0x219,
  kSiteDQEmpty = 0x21A,
  kSiteMmaDone = 0x21B,
  kSiteDSTmem = 0x21C,
  kSiteAccFree = 0x21D,
  kSiteKVFree = 0x21E,
};

// Block `blk` of the list of items: a key tile of a key head (from split_from
// on a part of its query tiles) and its query tiles i_first..i_last, head by head.
struct KeyItem {
  int bh, kt, k0;  // key head, key tile, its first key
  int part;        // of a split item, else -1
  int i_first, i_last;
  int n_iter;      // query tiles (all heads')
  int i, head;     // the first: tile and query head

  __device__ __forceinline__ void next() {
    if (++i > i_last) {
      i = i_first;
      ++head;
    }
  }
};

__device__ __forceinline__ KeyItem key_item(const BwdParams& p, int blk) {
  KeyItem t;
  t.part = -1;
  int item = blk;
  if (blk >= p.split_from) {
    const int i = p.div_parts.div(blk - p.split_from);
    item = p.split_from + i;
    t.part = blk - p.split_from - i * p.split_parts;
  }
  t.bh = p.div_kblk.div(item);
  t.kt = item - t.bh * p.n_kblk;
  t.k0 = t.kt * kBlockN;
  t.i_first = t.kt;
  // (window <= N <= 2^30, so the sum is an int)
  t.i_last = min((p.N + kBlockM - 1) / kBlockM - 1, (t.k0 + kBlockN - 2 + p.window) / kBlockM);
  const int per = t.i_last - t.i_first + 1;
  t.n_iter = p.group * per;
  int start = 0;
  if (t.part >= 0) {
    const int q = p.div_parts.div(t.n_iter), r = t.n_iter - q * p.split_parts;
    start = q * t.part + min(t.part, r);
    t.n_iter = q + (t.part < r ? 1 : 0);
  }
  t.head = t.bh * p.group;
  t.i = t.i_first;
  if (start > 0) {
    const int h = start / per;
    t.head += h;
    t.i += start - h * per;
  }
  return t;
}

// The next block from `blk` on, in steps of `stride`, that has query tiles (a
// part of a split item may have none); false if there is none.
__device__ __forceinline__ bool next_item(const BwdParams& p, int& blk, int stride, int total, KeyItem& t) {
  for (; blk < total; blk += stride) {
    t = key_item(p, blk);
    if (t.n_iter > 0) return true;
  }
  return false;
}

__global__ void __launch_bounds__(WinCfg::kThreads, 1)
    fa_bwd_window64_kernel(const __grid_constant__ BwdParams p) {
  using C = WinCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlotOff);
  const WaitCtl ctl{abort_flag, p.status};
  const int warp = warp_id();
  const int lane = lane_id();
  const int total = p.split_from + (p.n_kblk * p.BH - p.split_from) * p.split_parts;
  const int stride = static_cast<int>(gridDim.x);

  // One arrival for the warp's lanes, each of which has made its own fence: lanes
  // that all arrive take turns at the barrier's word, and shared memory is what
  // bounds this kernel.
  auto warp_arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  // m: the CTA's count of items that have query tiles
  auto load_kv = [&](int m, const KeyItem& t) {
    const int b = m & 1;
    mbar_arrive_expect_tx(bar(C::kBarKV + b), 2 * C::kTileBytes);
    tma_load_3d(sbase + C::kKOff + b * C::kTileBytes, &p.tm_k, bar(C::kBarKV + b), 0, t.k0, t.bh);
    tma_load_3d(sbase + C::kVOff + b * C::kTileBytes, &p.tm_v, bar(C::kBarKV + b), 0, t.k0, t.bh);
  };
  auto load_tile = [&](int s, const KeyItem& t) {
    mbar_arrive_expect_tx(bar(C::kBarStFull + s), 2 * C::kTileBytes);
    tma_load_3d(sbase + C::kQOff + s * C::kTileBytes, &p.tm_q, bar(C::kBarStFull + s), 0, t.i * kBlockM, t.head);
    tma_load_3d(sbase + C::kDOOff + s * C::kTileBytes, &p.tm_do, bar(C::kBarStFull + s), 0, t.i * kBlockM, t.head);
  };

  // the loader's thread initialises the barriers and starts the first item's
  // copies at once, beside the rest of the set-up
  if (threadIdx.x == C::kProducerWarp * 32) {
    *abort_flag = 0;
    mbar_init(bar(C::kBarKV), 1);
    mbar_init(bar(C::kBarKV + 1), 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarStFull + s), 2);
      mbar_init(bar(C::kBarStEmpty + s), 1);
    }
    mbar_init(bar(C::kBarSFull), 1);
    mbar_init(bar(C::kBarDPFull), 1);
    mbar_init(bar(C::kBarPFull), C::kComputeWarps);
    mbar_init(bar(C::kBarDSTmem), C::kComputeWarps);
    mbar_init(bar(C::kBarDSFull), C::kComputeWarps);
    mbar_init(bar(C::kBarDQFull), 1);
    mbar_init(bar(C::kBarDQEmpty), 4);
    mbar_init(bar(C::kBarMmaDone), 1);
    mbar_init(bar(C::kBarAccFree), C::kComputeWarps);
    mbar_init(bar(C::kBarKVFree), 2);
    fence_mbar_init();
    grid_dependency_wait();
    KeyItem t;
    int blk = blockIdx.x;
    if (next_item(p, blk, stride, total, t)) {
      load_kv(0, t);
      load_tile(0, t);
    }
  }
  if (warp == C::kMmaWarp) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();

  // Every role counts the CTA's query tiles (n) and the items that have some (m)
  // as it walks: the parities of the barriers.
  if (warp >= C::kProducerWarp) {
    regs_set<C::kOtherRegs, C::kLaunchRegs>();
    if (warp == C::kProducerWarp) {
      // ----------------------------------------------------------- loads
      int n = 0;
      bool ok = true;
      auto wait = [&](int b, uint32_t parity, unsigned int site) {
        ok = mbar_wait_short(bar(b), parity, ctl, site);
        return ok = __all_sync(0xffffffffu, ok);
      };
      int blk = blockIdx.x;
      KeyItem t;
      for (bool more = next_item(p, blk, stride, total, t); ok && more;) {
        for (int it = 0; it < t.n_iter; ++it) {
          const int s = n % C::kStages;
          // fp32 rows -LSE_q log2 e and -D_q; rows past N get -inf (P = 0 there)
          // and D = 0.  Read before the wait for the stage.
          const int q0 = t.i * kBlockM;
          const size_t head_row = static_cast<size_t>(t.head) * p.N;
          float nl[4], nd[4];
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            const int q = q0 + r4 * 32 + lane;
            nl[r4] = (q < p.N) ? -p.lse[head_row + q] * p.log2e : -INFINITY;
            nd[r4] = (q < p.N) ? -p.dsum[head_row + q] : 0.0f;
          }
          if (n >= C::kStages && !wait(C::kBarStEmpty + s, (n / C::kStages - 1) & 1, kSiteStEmpty)) break;
          if (lane == 0 && n > 0) load_tile(s, t);  // (the very first is on its way)
          float* row_l = reinterpret_cast<float*>(smem + C::kRowsOff + 2 * s * C::kRowBytes);
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            row_l[r4 * 32 + lane] = nl[r4];
            row_l[kBlockM + r4 * 32 + lane] = nd[r4];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBarStFull + s));
          ++n;
          t.next();
        }
        blk += stride;
        more = ok && next_item(p, blk, stride, total, t);
      }
      // Let every copy this CTA started land before shared memory is released
      // (only on the give-up path, where a barrier may lack the loader's own
      // arrival or have no copy in flight: the waits are bounded).
      if (lane == 0 && !ok) {
        for (int k = max(0, n - C::kStages); k < n; ++k)
          mbar_wait_drain(bar(C::kBarStFull + k % C::kStages), (k / C::kStages) & 1);
      }
    } else if (warp == C::kKVWarp && lane == 0) {
      // ----------------------------------------------------------- K and V
      bool ok = true;
      int blk = blockIdx.x;
      KeyItem t;
      bool more = next_item(p, blk, stride, total, t);  // (its copies are on their way)
      int m = 1;
      while (more) {
        blk += stride;
        more = next_item(p, blk, stride, total, t);
        if (!more) break;
        // the buffers are free once dV and dK of the item before the last have
        // left them
        if (m > 1 && !(ok = mbar_wait_short(bar(C::kBarKVFree), (m - 2) & 1, ctl, kSiteKVFree))) break;
        load_kv(m++, t);
      }
      if (!ok)
        for (int k = m - 2; k < m; ++k) mbar_wait_drain(bar(C::kBarKV + (k & 1)), (k / 2) & 1);
    } else if (warp == C::kMmaWarp) {
      // ----------------------------------------------------------- MMA issue
      // warp-uniform code (see fa_device.cuh): operand arithmetic in uniform
      // registers.  An N = 64 product is 32 cycles of the tensor core, and one lane's
      // own issue took 70 to 85.
      constexpr uint32_t kIdescSq = idesc_bf16_f32(kBlockN, kBlockM, false, false);  // S^T, dP^T
      constexpr uint32_t kIdescKV = idesc_bf16_f32(kBlockN, D, false, true);          // dV, dK
      constexpr uint32_t kIdescQ = idesc_bf16_f32(kBlockM, D, true, true);            // dQ
      auto k_smem = [&](int m) { return sbase + C::kKOff + (m & 1) * C::kTileBytes; };
      auto v_smem = [&](int m) { return sbase + C::kVOff + (m & 1) * C::kTileBytes; };
      // Products: loops that step the operand descriptors (by bytes >> 4).
      auto issue_nt = [&](uint32_t a0, uint32_t b0, uint32_t dcol) {
        uint64_t ad = sdesc_sw128(a0, 16, 1024), bd = sdesc_sw128(b0, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk, ad += 32 >> 4, bd += 32 >> 4)
          mma_ss<true>(tmem_base + dcol, ad, bd, kIdescSq, kk > 0 ? 1u : 0u);
      };
      auto issue_tn = [&](uint32_t acol, uint32_t b0, uint32_t dcol, bool accumulate) {
        uint64_t bd = sdesc_sw128(b0, C::kHalfBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kBlockM / 16; ++kk, bd += 2048 >> 4)
          mma_ts<true>(tmem_base + dcol, tmem_base + acol + C::packed_col(kk), bd, kIdescKV,
                       (accumulate || kk > 0) ? 1u : 0u);
      };
      auto issue_dq = [&](uint32_t ds0, uint32_t k0) {
        uint64_t dsd = sdesc_sw128(ds0, kBlockN * 128, 1024), kd = sdesc_sw128(k0, C::kHalfBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk, dsd += 2048 >> 4, kd += 2048 >> 4)
          mma_ss<true>(tmem_base + C::kColDQ, dsd, kd, kIdescQ, kk > 0 ? 1u : 0u);
      };
      // Step n issues tile n's dV, dK and dQ and tile n + 1's S^T and dP^T; step -1,
      // the first item's first S^T and dP^T alone.
      int m = 0, blk = blockIdx.x;
      KeyItem t;
      bool more = next_item(p, blk, stride, total, t);
      int left = 0, next_left = more ? t.n_iter : 0;  // tiles of the item from this step's on; of the next item
      bool first = false;                             // this step's tile is its item's first
      bool ok = true;
      for (int n = -1;; ++n) {
        const bool last = left <= 1;  // (of the item, or step -1)
        const bool next = !last || next_left > 0;
        if (n < 0 && !next) break;
        const int s = n % C::kStages;
        const int next_m = n >= 0 && last ? m + 1 : m;
        if (n >= 0) {
          if (!(ok = mbar_wait_short_warp(bar(C::kBarPFull), n & 1, ctl, kSitePFull))) break;
          if (first && m > 0 && !(ok = mbar_wait_short_warp(bar(C::kBarAccFree), (m - 1) & 1, ctl, kSiteAccFree))) break;
          tc_fence_after();
          issue_tn(C::kColS, sbase + C::kDOOff + s * C::kTileBytes, C::kColDV, !first);
        }
        // the next tile's S^T over P^T, which dV (issued before it) has read
        if (next) {
          const int s1 = (n + 1) % C::kStages;
          if (last && !(ok = mbar_wait_short_warp(bar(C::kBarKV + (next_m & 1)), (next_m / 2) & 1, ctl, kSiteKV))) break;
          if (!(ok = mbar_wait_short_warp(bar(C::kBarStFull + s1), ((n + 1) / C::kStages) & 1, ctl, kSiteStFull))) break;
          tc_fence_after();
          issue_nt(k_smem(next_m), sbase + C::kQOff + s1 * C::kTileBytes, C::kColS);
          mma_commit<true>(bar(C::kBarSFull));
        }
        if (n >= 0) {
          if (!(ok = mbar_wait_short_warp(bar(C::kBarDSTmem), n & 1, ctl, kSiteDSTmem))) break;
          tc_fence_after();
          issue_tn(C::kColDP, sbase + C::kQOff + s * C::kTileBytes, C::kColDK, !first);
          mma_commit<true>(bar(C::kBarStEmpty + s));  // the last to read the stage
        }
        if (next) {  // over dS^T
          issue_nt(v_smem(next_m), sbase + C::kDOOff + ((n + 1) % C::kStages) * C::kTileBytes, C::kColDP);
          mma_commit<true>(bar(C::kBarDPFull));
        }
        if (n >= 0) {
          if (!(ok = mbar_wait_short_warp(bar(C::kBarDSFull), n & 1, ctl, kSiteDSFull))) break;
          if (n > 0 && !(ok = mbar_wait_short_warp(bar(C::kBarDQEmpty), (n - 1) & 1, ctl, kSiteDQEmpty))) break;
          tc_fence_after();
          issue_dq(sbase + C::kDsOff, k_smem(m));
          mma_commit<true>(bar(C::kBarDQFull));
          if (last) {
            mma_commit<true>(bar(C::kBarMmaDone));
            ++m;
          }
        }
        if (!next) break;
        first = last;
        --left;
        if (last) {
          left = next_left;
          blk += stride;
          next_left = next_item(p, blk, stride, total, t) ? t.n_iter : 0;
        }
      }
      if (!ok) {
        // what was issued finishes before tensor memory is freed
        mma_commit<true>(bar(C::kBarMmaDone));
        mbar_wait_drain(bar(C::kBarMmaDone), m & 1);
      } else if (m > 0) {
        mbar_wait_short_warp(bar(C::kBarMmaDone), (m - 1) & 1, ctl, kSiteMmaDone);
      }
    }
  } else if (warp >= C::kDrainWarp0) {
    regs_set<C::kDrainRegs, C::kLaunchRegs>();
    // ------------------------------------------------------------- dQ drain
    const int quarter = warp & 3;
    const int qr = quarter * 32 + lane;  // query row within the tile (d = 64)
    const bool leader = (warp == C::kDrainWarp0 && lane == 0);
    const uint32_t t_dq = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + C::kColDQ;
    int n = 0, buf = 0;
    bool ok = true;
    int blk = blockIdx.x;
    KeyItem t;
    for (; ok && next_item(p, blk, stride, total, t); blk += stride) {
      for (int it = 0; it < t.n_iter; ++it, ++n, t.next()) {
        ok = mbar_wait_short(bar(C::kBarDQFull), n & 1, ctl, kSiteDQFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          // release drain warps already waiting at this tile's barriers below (the
          // next tile's dQ never comes without this warp's kBarDQEmpty)
          for (int c = 0; c < C::kDqChunks; ++c) named_bar_arrive(C::kDrainBarrier, kBlockM);
          break;
        }
        tc_fence_after();
        const int q0 = t.i * kBlockM;
        uint32_t r[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16(t_dq + c * C::kDqCols, r[c]);
        tmem_ld_wait16(r[0]);
        reg_fence16(r[1]);
        reg_fence16(r[2]);
        reg_fence16(r[3]);
        tc_fence_before();
        warp_arrive(bar(C::kBarDQEmpty));
        // The fp32 dQ tile goes out in chunks of 16 columns (64-byte swizzled rows)
        // through a ring of buffers; the TMA adds them into the accumulator.
#pragma unroll
        for (int c = 0; c < C::kDqChunks; ++c) {
          uint8_t* chunk = smem + C::kDqOff + buf * C::kDqChunkBytes;
          uint8_t* row = chunk + qr * 64;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4)
            *reinterpret_cast<uint4*>(row + ((c4 ^ ((qr >> 1) & 3)) << 4)) =
                make_uint4(r[c][4 * c4], r[c][4 * c4 + 1], r[c][4 * c4 + 2], r[c][4 * c4 + 3]);
          fence_proxy_async_smem();
          // The leader comes to it once the TMA has read all chunks but the last
          // issued: the buffer written after the barrier is free.
          named_bar_sync(C::kDrainBarrier, kBlockM);
          if (leader) {
            tma_reduce_add_3d(&p.tm_dq, smem_u32(chunk), c * C::kDqCols, q0, t.head);
            bulk_commit();
            bulk_wait_read<1>();
          }
          buf = buf == C::kDqBufs - 1 ? 0 : buf + 1;
        }
      }
    }
    if (leader) bulk_wait<0>();
  } else {
    regs_set<C::kComputeRegs, C::kLaunchRegs>();
    // ------------------------------------------------------------- compute
    const int wg = warp >> 2;  // query-column half
    const int quarter = warp & 3;
    const int kr = quarter * 32 + lane;  // key row within the tile
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const f32x2 c2 = f2_pack(p.c, p.c);
    bool storing = false;  // this warpgroup's last dV or dK may still be in its buffer
    // its leader, once the TMA has read the buffer: the KV warp may load into it
    auto release = [&] {
      if (storing && kr == 0) {
        bulk_wait_read<0>();
        mbar_arrive(bar(C::kBarKVFree));
      }
      storing = false;
    };
    int n = 0, m = 0;
    bool ok = true;
    KeyItem t_next;
    if (static_cast<int>(blockIdx.x) < total) t_next = key_item(p, blockIdx.x);
    for (int blk = blockIdx.x; ok && blk < total; blk += stride) {
      KeyItem t = t_next;
      const bool row_valid = t.k0 + kr < p.N;
      const bool last_tile = t.k0 + kBlockN > p.N;  // some key rows are past N
      for (int it = 0; it < t.n_iter; ++it, ++n, t.next()) {
        const int s = n % C::kStages;
        // the diagonal tile, those whose last rows are past some key's window,
        // and all of a key tile with rows past N
        const bool edge = t.i == t.kt || (t.i - t.kt) * kBlockM + kBlockM - 1 >= p.window || last_tile;
        ok = mbar_wait_short(bar(C::kBarSFull), n & 1, ctl, kSiteSFull);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        // returns at once (S^T was issued after the stage landed); makes the
        // loader's rows visible
        ok = mbar_wait_short(bar(C::kBarStFull + s), (n / C::kStages) & 1, ctl, kSiteStFull);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        // this warpgroup's 64 queries' -LSE log2 e and -D
        const float4* rl4 = reinterpret_cast<const float4*>(smem + C::kRowsOff + 2 * s * C::kRowBytes) + wg * 16;
        const float4* rd4 = rl4 + kBlockM / 4;
        uint32_t sr[2][32];  // S, then P in fp32
        tmem_ld32(lane_base + C::kColS + wg * 64, sr[0]);
        tmem_ld32(lane_base + C::kColS + wg * 64 + 32, sr[1]);
        tmem_ld_wait(sr[0]);
        reg_fence(sr[1]);
        auto exp_pair = [&](int ch, int e2, float& p0, float& p1) {
          const f32x2 x = f2_pack(__uint_as_float(sr[ch][2 * e2]), __uint_as_float(sr[ch][2 * e2 + 1]));
          const float4 l4 = rl4[ch * 8 + (e2 >> 1)];
          float x0, x1;
          f2_unpack(f2_fma(x, c2, (e2 & 1) ? f2_pack(l4.z, l4.w) : f2_pack(l4.x, l4.y)), x0, x1);
          p0 = ex2_mufu(x0);
          p1 = ex2_mufu(x1);
        };
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) {
            float p0, p1;
            exp_pair(ch, e2, p0, p1);
            sr[ch][2 * e2] = __float_as_uint(p0);
            sr[ch][2 * e2 + 1] = __float_as_uint(p1);
          }
        if (edge) {
          // the key sees the query columns [lo, lo + window) of the tile
          const int lo = (t.kt - t.i) * kBlockM + kr - wg * 64;
          const int hi = lo + p.window;
          auto below = [](int k) { return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u; };
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t seen = row_valid ? below(hi - ch * 32) & ~below(lo - ch * 32) : 0u;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen & (1u << e))) sr[ch][e] = 0u;
          }
        }
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t w[16];
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2)
            w[e2] = pack_bf16x2(__uint_as_float(sr[ch][2 * e2]), __uint_as_float(sr[ch][2 * e2 + 1]));
          tmem_st16(lane_base + C::kColS + wg * 64 + ch * 16, w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::kBarPFull));
        release();

        // dS = P (dP - D)^T (unscaled): to tensor memory (for dK) and shared
        // memory (for dQ)
        ok = mbar_wait_short(bar(C::kBarDPFull), n & 1, ctl, kSiteDPFull);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        uint32_t dsw[32];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t dr[32];
          tmem_ld32(lane_base + C::kColDP + wg * 64 + ch * 32, dr);
          tmem_ld_wait(dr);
          uint32_t w[16];
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) {
            const float4 d4 = rd4[ch * 8 + (e2 >> 1)];
            const f32x2 dp = f2_add(f2_pack(__uint_as_float(dr[2 * e2]), __uint_as_float(dr[2 * e2 + 1])),
                                    (e2 & 1) ? f2_pack(d4.z, d4.w) : f2_pack(d4.x, d4.y));
            float a0, a1;
            f2_unpack(f2_mul(dp, f2_pack(__uint_as_float(sr[ch][2 * e2]), __uint_as_float(sr[ch][2 * e2 + 1]))), a0, a1);
            w[e2] = dsw[ch * 16 + e2] = pack_bf16x2(a0, a1);
          }
          tmem_st16(lane_base + C::kColDP + wg * 64 + ch * 16, w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::kBarDSTmem));
        // dQ of the tile before has read the buffer
        if (n > 0) {
          ok = mbar_wait_short(bar(C::kBarDQFull), (n - 1) & 1, ctl, kSiteDQFull);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        // [query half][key row][64 queries], 16-byte chunk index XOR (key row mod 8)
        uint8_t* ds_tile = smem + C::kDsOff + wg * (kBlockN * 128) + kr * 128;
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8)
          *reinterpret_cast<uint4*>(ds_tile + ((c8 ^ (kr & 7)) << 4)) =
              make_uint4(dsw[4 * c8], dsw[4 * c8 + 1], dsw[4 * c8 + 2], dsw[4 * c8 + 3]);
        fence_proxy_async_smem();
        warp_arrive(bar(C::kBarDSFull));
      }
      if (blk + stride < total) t_next = key_item(p, blk + stride);

      // The item's dV (warpgroup 0) and dK (warpgroup 1, times the softmax scale,
      // which dS left out): a thread holds its key row.
      // A row that is joined in fp32 afterwards is written as such (unscaled): all
      // of a part's (zeros if it has no query tile), and the first tokens', which
      // also get the queries whose windows have left them.
      float* raw = nullptr;
      if (t.part >= 0)
        raw = p.tile_part + ((static_cast<size_t>(blk - p.split_from) * 2 + (wg == 0 ? 1 : 0)) * kBlockN + kr) * D;
      else if (p.sink_main != nullptr && t.kt == 0 && kr < p.sinks)
        raw = p.sink_main + ((static_cast<size_t>(t.bh) * 2 + (wg == 0 ? 1 : 0)) * p.sink_rows + kr) * D;
      if (ok && t.n_iter > 0) {
        ok = mbar_wait_short(bar(C::kBarMmaDone), m & 1, ctl, kSiteMmaDone);
        ok = __all_sync(0xffffffffu, ok);
      }
      // the warpgroup goes on, or gives up, together: its warps meet below
      if (!(ok = named_bar_and(C::kEpiBarrier0 + wg, kBlockM, ok))) break;
      uint32_t r[2][32];
      if (t.n_iter > 0) {
        tc_fence_after();
        const uint32_t col = wg == 0 ? C::kColDV : C::kColDK;
        tmem_ld32(lane_base + col, r[0]);
        tmem_ld32(lane_base + col + 32, r[1]);
        tmem_ld_wait(r[0]);
        reg_fence(r[1]);
        // dV and dK have left tensor memory: the next item may write them
        tc_fence_before();
        warp_arrive(bar(C::kBarAccFree));
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) r[0][e] = r[1][e] = 0u;
      }
      if (raw != nullptr) {
        float4* dst = reinterpret_cast<float4*>(raw);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t* x = &r[c >> 3][(c & 7) * 4];
          dst[c] = make_float4(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]),
                               __uint_as_float(x[3]));
        }
      }
      if (t.part < 0) {
        // as bf16 over the item's V or K, which its products were the last to read,
        // and out by TMA
        const float mul = wg == 0 ? 1.0f : p.scale;
        const int off = (wg == 0 ? C::kVOff : C::kKOff) + (m & 1) * C::kTileBytes;
        uint8_t* row = smem + off + kr * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t* x = &r[c >> 2][(c & 3) * 8];
          *reinterpret_cast<uint4*>(row + ((c ^ (kr & 7)) << 4)) =
              make_uint4(pack_bf16x2(__uint_as_float(x[0]) * mul, __uint_as_float(x[1]) * mul),
                         pack_bf16x2(__uint_as_float(x[2]) * mul, __uint_as_float(x[3]) * mul),
                         pack_bf16x2(__uint_as_float(x[4]) * mul, __uint_as_float(x[5]) * mul),
                         pack_bf16x2(__uint_as_float(x[6]) * mul, __uint_as_float(x[7]) * mul));
        }
        fence_proxy_async_smem();
        named_bar_sync(C::kEpiBarrier0 + wg, kBlockM);
        if (kr == 0) {
          tma_store_3d(wg == 0 ? &p.tm_dv : &p.tm_dk, sbase + off, 0, t.k0, t.bh);
          bulk_commit();
        }
      }
      if (t.n_iter > 0) {
        storing = true;
        ++m;
      }
    }
    release();
  }

  tc_fence_before();
  __syncthreads();
  record_abort(ctl);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace

cudaError_t launch_bwd_window64(const BwdParams& p, cudaStream_t stream) {
  using C = WinCfg;
  cudaError_t err = configure_kernel<fa_bwd_window64_kernel>(C::kSmemBytes, C::kLaunchRegs);
  if (err != cudaSuccess) return err;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int total = p.split_from + (p.n_kblk * p.BH - p.split_from) * p.split_parts;
  err = launch_dependent(fa_bwd_window64_kernel, dim3(static_cast<unsigned int>(total < sms ? total : sms)),
                         dim3(C::kThreads), C::kSmemBytes, stream, p);
  if (err != cudaSuccess) return err;
  return launched(1);
}

}  // namespace fa
