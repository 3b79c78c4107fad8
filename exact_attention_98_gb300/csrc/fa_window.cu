// The first tokens' share of the sliding-window backward.
//
// The main kernel (fa_bwd_window_kernel) walks, key tile by key tile, the
// query tiles whose windows reach it.  The few first tokens are also seen by
// every later query, whose windows have left them: a key-stationary CTA
// would walk all of these for a tile of 128 keys of which a handful
// count.  Those pairs (query i, key j < sinks, j <= i - window) are computed here
// instead, beside D = rowsum(dO * O), which has to read O and dO anyway: this
// kernel reads Q besides, and writes its dQ as the accumulator's start where the
// plain backward writes zeros.  With 16 keys a row costs about
// 10 * 16 * d flops for 10 d bytes, so it is bound by HBM; the products are
// m16n8k16 mma.sync, whose operands never leave registers (up to 8 first tokens:
// NT = 1, half the columns and half the registers of dK_s and dV_s):
//   S = Q K_s^T, dP = dO V_s^T, P = exp2(c S - LSE log2 e), dS = P (dP - D),
//   dQ = dS K_s, dK_s += dS^T Q, dV_s += P^T dO
// (dS without the softmax scale, as in the main kernel).  dS and the P of the dV
// product are rounded to bf16, as there.  The lanes of a quad take d in
// runs of D/4, so that Q, dO and O are read 16 bytes at a time.
//
// Rows come by bulk copies into a ring in shared memory, one tile of 16 ahead (88
// -> 69 us: plain loads left too few bytes in flight at two CTAs of 4 warps per SM),
// and are read with few bank conflicts (61).  Measured (B = 2, H = 16, Hkv = 4, N =
// 8192, d = 128, 4 first tokens; 202 MB read, 134 MB written): 61 us, 5.5 TB/s;
// shared memory's wavefronts are at 68%, DRAM at 57% under a profiler.
//
// A key head's queries are cut into parts, each with dK_s and dV_s of its own;
// the kernel after the main one adds the parts and the main kernel's rows in a
// fixed order, so dK and dV have the same bits from run to run.
#include "fa_device.cuh"
#include "fa_kernels.h"

namespace fa {
namespace {

constexpr int kWarps = 4;

enum : unsigned int {
  kSiteWindowTile = 0x601,
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int D, int NT>
struct PreCfg {
  static constexpr int kKeys = 8 * NT;  // keys of a pass
  static constexpr int kPitch = D + 8;  // of a key row in shared memory: no bank conflicts
  static constexpr int kStages = 2;
  static constexpr int kTileBytes = 16 * D * 2;  // 16 rows of Q, dO or O: contiguous
  static constexpr int kStageBytes = 3 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kKOff = kRingBytes;
  static constexpr int kVOff = kKOff + kKeys * kPitch * 2;
  static constexpr int kBarOff = kVOff + kKeys * kPitch * 2;
  static constexpr int kAbortOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kSmemBytes = kAbortOff + 16;
  static_assert(kWarps * kKeys * D * 4 <= kRingBytes, "the warps' sums go over the ring");
};

// grid slots * BHkv.  A warp takes 16 rows of one query head at a time; lane
// (g, c) their rows g and g + 8, and of each the elements [c D/4, (c+1) D/4).
// The next 16 rows are on their way into the warp's ring meanwhile.
// NT: tiles of 8 first tokens in a pass over the rows.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps) fa_window_pre_kernel(const __grid_constant__ WindowParams p) {
  using C = PreCfg<D, NT>;
  constexpr int kSteps = D / 16;
  constexpr int kKeys = C::kKeys, kPitch = C::kPitch;
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16* ks = reinterpret_cast<__nv_bfloat16*>(smem + C::kKOff);
  __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(smem + C::kVOff);
  float (*sum)[kKeys][D] = reinterpret_cast<float (*)[kKeys][D]>(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);
  const WaitCtl ctl{abort_flag, p.status};
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, c = lane & 3;
  // lanes with c >= 2 take their run's 16-byte chunks in pairs exchanged: the four
  // lanes of a quad, D/2 bytes apart, would meet in the same banks otherwise
  const int turn = c >> 1;
  const int slot = blockIdx.x % p.slots, bkv = blockIdx.x / p.slots;
  const uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_s = smem_u32(ring);
  const uint32_t bars = smem_u32(smem + C::kBarOff) + warp * C::kStages * 8;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kWarps * C::kStages; ++i) mbar_init(smem_u32(smem + C::kBarOff) + 8 * i, 1);
    fence_mbar_init();
  }
  grid_dependency_wait();

  const int row_begin = slot * p.slot_rows;
  const int row_end = min(p.N, row_begin + p.slot_rows);
  // 16-row tiles of the part, of each head of the group in turn
  const int per_head = (row_end - row_begin + 15) / 16, tiles = per_head * p.group;
  const FastDiv div_tiles = row_end - row_begin == p.slot_rows ? p.div_tiles : p.div_last_tiles;
  int stage = 0;          // of the next tile to use
  uint32_t parity = 0;    // of its barrier
  int issue_stage = 0;
  bool ok = true;
  for (int key0 = 0; key0 < p.sinks; key0 += kKeys) {
    fence_proxy_async_smem();  // the sums of the pass before, written over the ring, before the copies into it
    __syncthreads();  // the pass before has read ks, vs and sum; the barriers are initialised
    for (int i = threadIdx.x; i < kKeys * D / 8; i += 32 * kWarps) {
      const int r = i / (D / 8), col = (i % (D / 8)) * 8;
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (key0 + r < p.sinks) {
        const size_t at = (static_cast<size_t>(bkv) * p.N + key0 + r) * D + col;
        a = *reinterpret_cast<const uint4*>(p.k + at);
        b = *reinterpret_cast<const uint4*>(p.v + at);
      }
      *reinterpret_cast<uint4*>(ks + r * kPitch + col) = a;
      *reinterpret_cast<uint4*>(vs + r * kPitch + col) = b;
    }
    __syncthreads();
    // dK_s^T and dV_s^T: keys 8 nt + 2c + {0, 1} (e & 1) at d(g) + 4 (k ^ 2 (g / 4))
    // (+ 2 for e >> 1), d(g) = (g / 2) D/4 + g % 2
    float dk[kSteps][NT][4], dv[kSteps][NT][4];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[k][nt][e] = dv[k][nt][e] = 0.0f;

    auto first_row = [&](int t) { return row_begin + (t - div_tiles.div(t) * per_head) * 16; };
    // any pair of the 16 rows from r0 with keys of this pass?
    auto is_far = [&](int r0) { return min(r0 + 15, p.N - 1) - key0 >= p.window; };
    // the tile from t on that this pass has to read
    auto needed = [&](int t) {
      if (key0 > 0)
        while (t < tiles && !is_far(first_row(t))) t += kWarps;
      return t;
    };
    auto issue = [&](int t) {
      if (t >= tiles) return;
      const int r0 = first_row(t);
      const uint32_t bytes = static_cast<uint32_t>(min(16, p.N - r0)) * D * 2;
      const size_t at = ((static_cast<size_t>(bkv) * p.group + div_tiles.div(t)) * p.N + r0) * D;
      const bool far = is_far(r0);
      if (lane == 0) {
        const uint32_t dst = ring_s + issue_stage * C::kStageBytes, bar = bars + 8 * issue_stage;
        mbar_arrive_expect_tx(bar, bytes * (1u + (far ? 1u : 0u) + (key0 == 0 ? 1u : 0u)));
        if (far) bulk_load(dst, p.q + at, bytes, bar);
        bulk_load(dst + C::kTileBytes, p.dout + at, bytes, bar);
        if (key0 == 0) bulk_load(dst + 2 * C::kTileBytes, p.o + at, bytes, bar);
      }
      issue_stage ^= 1;
    };
    int ahead = needed(warp);  // the next tile to copy
    for (int i = 0; i < C::kStages; ++i) {
      if (ok) issue(ahead);
      ahead = needed(ahead + kWarps);
    }
    {
      for (int t = needed(warp); t < tiles; t = needed(t + kWarps)) {
        const int r0 = first_row(t);
        const size_t head_row = (static_cast<size_t>(bkv) * p.group + div_tiles.div(t)) * p.N;
        const bool far = is_far(r0);
        const uint8_t* st = ring + stage * C::kStageBytes;
        if (ok && !mbar_wait_warp(bars + 8 * stage, parity, ctl, kSiteWindowTile)) {
          // given up: no more copies; those in flight land before shared memory
          // is released
          ok = false;
          for (int i = 0; i < C::kStages; ++i)
            mbar_wait_drain(bars + 8 * ((stage + i) % C::kStages), parity ^ (stage + i >= C::kStages ? 1u : 0u));
        }
        uint32_t qa[kSteps][4], da[kSteps][4];
        float dsum[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = r0 + g + 8 * r;
          const bool in = row < p.N;
          const uint4* at = reinterpret_cast<const uint4*>(st + (g + 8 * r) * (D * 2) + c * (D / 2));
          dsum[r] = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (in) y = at[C::kTileBytes / 16 + (i ^ turn)];
            if (in && far) x = at[i ^ turn];
            qa[2 * i][r] = x.x; qa[2 * i][2 + r] = x.y; qa[2 * i + 1][r] = x.z; qa[2 * i + 1][2 + r] = x.w;
            da[2 * i][r] = y.x; da[2 * i][2 + r] = y.y; da[2 * i + 1][r] = y.z; da[2 * i + 1][2 + r] = y.w;
            if (key0 == 0) {
              uint4 o = make_uint4(0u, 0u, 0u, 0u);
              if (in) o = at[2 * (C::kTileBytes / 16) + (i ^ turn)];
              const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                dsum[r] = fmaf(bf16_lo(ow[e]), bf16_lo(yw[e]), dsum[r]);
                dsum[r] = fmaf(bf16_hi(ow[e]), bf16_hi(yw[e]), dsum[r]);
              }
            }
          }
          if (key0 == 0) {
            dsum[r] += __shfl_xor_sync(0xffffffffu, dsum[r], 1);
            dsum[r] += __shfl_xor_sync(0xffffffffu, dsum[r], 2);
            if (in && c == 0) p.dsum[head_row + row] = dsum[r];
          } else {
            dsum[r] = in ? p.dsum[head_row + row] : 0.0f;  // written by this block in its first pass
          }
        }
        __syncwarp();  // every lane has read the stage
        if (ok) issue(ahead);
        ahead = needed(ahead + kWarps);
        if (++stage == C::kStages) {
          stage = 0;
          parity ^= 1u;
        }
        float* acc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) acc[r] = p.dq_acc + (head_row + r0 + g + 8 * r) * D + 2 * c;
        const bool in0 = r0 + g < p.N, in1 = r0 + g + 8 < p.N;
        if (!far) {
#pragma unroll
          for (int j = 0; j < 2 * kSteps; ++j) {
            if (in0) *reinterpret_cast<float2*>(acc[0] + 8 * j) = make_float2(0.0f, 0.0f);
            if (in1) *reinterpret_cast<float2*>(acc[1] + 8 * j) = make_float2(0.0f, 0.0f);
          }
          continue;
        }
        // S and dP: key key0 + 8 nt + 2c + {0, 1} of rows g (0, 1) and g + 8 (2, 3)
        float s[NT][4], dp[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = dp[nt][e] = 0.0f;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int at = (nt * 8 + g) * kPitch + c * (D / 4) + 4 * (k ^ (2 * turn));
            const uint2 kk = *reinterpret_cast<const uint2*>(ks + at);
            const uint2 vv = *reinterpret_cast<const uint2*>(vs + at);
            mma_bf16(s[nt], qa[k], kk.x, kk.y);
            mma_bf16(dp[nt], da[k], vv.x, vv.y);
          }
        }
        uint32_t pp[NT][2], dd[NT][2];  // P and dS as bf16 pairs: [nt][row]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = r0 + g + 8 * r;
          const float lse = row < p.N ? p.lse[head_row + row] * p.log2e : 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pe[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + nt * 8 + 2 * c + e;
              const bool seen = key < p.sinks && row - key >= p.window && row < p.N;
              pe[e] = seen ? ex2_mufu(fmaf(s[nt][2 * r + e], p.c, -lse)) : 0.0f;
            }
            pp[nt][r] = pack_bf16x2(pe[0], pe[1]);
            dd[nt][r] = pack_bf16x2(pe[0] * (dp[nt][2 * r] - dsum[r]), pe[1] * (dp[nt][2 * r + 1] - dsum[r]));
          }
        }
        // dQ = dS K_s (d in order), 16 columns at a time
#pragma unroll
        for (int j = 0; j < 2 * kSteps; j += 2) {
          uint32_t b[2 * NT];  // keys 0-7 (and 8-15) of columns 8j.., then of the next 8
          const uint32_t row_s =
              smem_u32(ks) + (NT == 2 ? (lane & 15) * kPitch + (lane >> 4) * 8 : (lane & 7) * kPitch + ((lane >> 3) & 1) * 8) * 2;
          if constexpr (NT == 2)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                         : "r"(row_s + j * 16)
                         : "memory");
          else
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                         : "=r"(b[0]), "=r"(b[1])
                         : "r"(row_s + j * 16)
                         : "memory");
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (key0 > 0) {
              const float2 y0 = in0 ? *reinterpret_cast<const float2*>(acc[0] + 8 * (j + u)) : make_float2(0.f, 0.f);
              const float2 y1 = in1 ? *reinterpret_cast<const float2*>(acc[1] + 8 * (j + u)) : make_float2(0.f, 0.f);
              x[0] = y0.x; x[1] = y0.y; x[2] = y1.x; x[3] = y1.y;
            }
            if constexpr (NT == 2) {
              const uint32_t a[4] = {dd[0][0], dd[0][1], dd[1][0], dd[1][1]};
              mma_bf16(x, a, b[2 * u], b[2 * u + 1]);
            } else {
              mma_bf16_k8(x, dd[0][0], dd[0][1], b[u]);
            }
            if (in0) *reinterpret_cast<float2*>(acc[0] + 8 * (j + u)) = make_float2(x[0], x[1]);
            if (in1) *reinterpret_cast<float2*>(acc[1] + 8 * (j + u)) = make_float2(x[2], x[3]);
          }
        }
        // dK_s^T += Q^T dS, dV_s^T += dO^T P: 16 elements of d by 8 keys
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            dd[nt][r] = transpose8x8(dd[nt][r]);
            pp[nt][r] = transpose8x8(pp[nt][r]);
          }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint32_t qt[4] = {transpose8x8(qa[k][0]), transpose8x8(qa[k][2]), transpose8x8(qa[k][1]),
                                  transpose8x8(qa[k][3])};
          const uint32_t dt[4] = {transpose8x8(da[k][0]), transpose8x8(da[k][2]), transpose8x8(da[k][1]),
                                  transpose8x8(da[k][3])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(dk[k][nt], qt, dd[nt][0], dd[nt][1]);
            mma_bf16(dv[k][nt], dt, pp[nt][0], pp[nt][1]);
          }
        }
      }
    }

    // the four warps' dK_s, then dV_s, added in order (over the ring: every copy
    // has been waited for)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum[warp][nt * 8 + 2 * c + (e & 1)]
               [(g >> 1) * (D / 4) + 4 * (k ^ (2 * (g >> 2))) + 2 * (e >> 1) + (g & 1)] =
                which == 0 ? dk[k][nt][e] : dv[k][nt][e];
      __syncthreads();
      float* out = p.sink_part + (((static_cast<size_t>(slot) * p.BHkv + bkv) * 2 + which) * p.sink_rows + key0) * D;
      for (int i = threadIdx.x * 4; i < kKeys * D; i += 32 * kWarps * 4) {
        float4 x = *reinterpret_cast<const float4*>(&sum[0][0][0] + i);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(&sum[w][0][0] + i);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        *reinterpret_cast<float4*>(out + i) = x;
      }
    }
  }
}

// After the main kernel, three kinds of blocks:
//   sink_blocks      a first token's row of dK (times the softmax scale) or dV
//                    from all its parts; the thread groups take every
//                    kGroups-th part
//   tile_blocks      16 rows of a split item's dK or dV from its parts
//   the others       dQ = scale * its accumulator, as bf16, 32 elements a thread
//                    per step, all loads first
template <int D>
__global__ void __launch_bounds__(256) fa_window_post_kernel(const __grid_constant__ WindowParams p) {
  constexpr int kGroups = 256 / D;
  __shared__ float part[kGroups][D];
  grid_dependency_wait();
  int blk = static_cast<int>(blockIdx.x);
  if (blk < p.sink_blocks) {
    const int col = threadIdx.x % D, grp = threadIdx.x / D;
    const int key = blk % p.sinks, which = (blk / p.sinks) & 1, bkv = blk / p.sinks / 2;
    const size_t stride = static_cast<size_t>(p.BHkv) * 2 * p.sink_rows * D;
    const float* from = p.sink_part + ((static_cast<size_t>(bkv) * 2 + which) * p.sink_rows + key) * D + col;
    const int item = bkv * p.n_kblk;  // its first key tile
    const bool split = item >= p.split_from;
    float x = 0.0f;
#pragma unroll 8
    for (int s = grp; s < p.slots + (split ? 0 : 1); s += kGroups) x += from[s * stride];
    if (split)
      for (int k = grp; k < p.split_parts; k += kGroups)
        x += p.tile_part[((static_cast<size_t>(item - p.split_from) * p.split_parts + k) * 2 + which) * kBlockN * D +
                         key * D + col];
    part[grp][col] = x;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < kGroups; ++k) x += part[k][col];
    __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N + key) * D + col;
    *out = __float2bfloat16_rn(which == 0 ? x * p.scale : x);
    return;
  }
  blk -= p.sink_blocks;
  if (blk < p.tile_blocks) {
    constexpr int kRows = 16, kPerTile = kBlockN / kRows;
    const int which = (blk / kPerTile) & 1, rel = blk / kPerTile / 2, row0 = blk % kPerTile * kRows;
    const int item = p.split_from + rel;
    const int bkv = item / p.n_kblk, key0 = item % p.n_kblk * kBlockN + row0;
    const float mul = which == 0 ? p.scale : 1.0f;
    const float4* from = reinterpret_cast<const float4*>(p.tile_part) +
                         ((static_cast<size_t>(rel) * p.split_parts * 2 + which) * kBlockN + row0) * (D / 4);
    __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N + key0) * D;
    for (int i = threadIdx.x; i < kRows * D / 4; i += 256) {
      const int key = key0 + i / (D / 4);
      if (key >= p.N || (p.sink_blocks > 0 && key < p.sinks)) continue;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < p.split_parts; ++k) {
        const float4 y = from[static_cast<size_t>(k) * 2 * kBlockN * (D / 4) + i];
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16x2(x.x * mul, x.y * mul), pack_bf16x2(x.z * mul, x.w * mul));
    }
    return;
  }
  blk -= p.tile_blocks;
  const long long n8 = static_cast<long long>(p.BHkv) * p.group * p.N * (D / 8);
  const long long stride = static_cast<long long>(gridDim.x - p.sink_blocks - p.tile_blocks) * 256;
  for (long long i0 = blk * 256LL + threadIdx.x; i0 < n8; i0 += 4 * stride) {
    float4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = i0 + u * stride;
      if (i < n8) {
        a[u] = reinterpret_cast<const float4*>(p.dq_acc)[2 * i];
        b[u] = reinterpret_cast<const float4*>(p.dq_acc)[2 * i + 1];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = i0 + u * stride;
      if (i < n8)
        reinterpret_cast<uint4*>(p.dq)[i] =
            make_uint4(pack_bf16x2(a[u].x * p.scale, a[u].y * p.scale), pack_bf16x2(a[u].z * p.scale, a[u].w * p.scale),
                       pack_bf16x2(b[u].x * p.scale, b[u].y * p.scale), pack_bf16x2(b[u].z * p.scale, b[u].w * p.scale));
    }
  }
}

}  // namespace

cudaError_t launch_window_pre(const WindowParams& p, int d, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned int>(p.slots) * static_cast<unsigned int>(p.BHkv));
  // up to 8 first tokens: half the accumulators, so more warps per SM
  auto kernel = p.sinks <= 8 ? (d == 128 ? fa_window_pre_kernel<128, 1> : fa_window_pre_kernel<64, 1>)
                             : (d == 128 ? fa_window_pre_kernel<128, 2> : fa_window_pre_kernel<64, 2>);
  const int smem = p.sinks <= 8 ? (d == 128 ? PreCfg<128, 1>::kSmemBytes : PreCfg<64, 1>::kSmemBytes)
                                : (d == 128 ? PreCfg<128, 2>::kSmemBytes : PreCfg<64, 2>::kSmemBytes);
  cudaError_t err = p.sinks <= 8 ? (d == 128 ? configure_kernel<fa_window_pre_kernel<128, 1>>(smem)
                                             : configure_kernel<fa_window_pre_kernel<64, 1>>(smem))
                                 : (d == 128 ? configure_kernel<fa_window_pre_kernel<128, 2>>(smem)
                                             : configure_kernel<fa_window_pre_kernel<64, 2>>(smem));
  if (err != cudaSuccess) return err;
  err = launch_dependent(kernel, grid, dim3(32 * kWarps), smem, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_window_post(WindowParams p, int d, cudaStream_t stream) {
  p.sink_blocks = p.slots > 0 ? p.sinks * 2 * p.BHkv : 0;
  p.tile_blocks = (p.n_kblk * p.BHkv - p.split_from) * 2 * (kBlockN / 16);
  const long long n8 = static_cast<long long>(p.BHkv) * p.group * p.N * (d / 8);
  const long long blocks = (n8 + 255) / 256, cap = (sm_count() > 0 ? sm_count() : 1) * 16LL;
  const dim3 grid(static_cast<unsigned int>(p.sink_blocks) + static_cast<unsigned int>(p.tile_blocks) +
                  static_cast<unsigned int>(blocks < cap ? blocks : cap));
  const cudaError_t err = launch_dependent(d == 128 ? fa_window_post_kernel<128> : fa_window_post_kernel<64>, grid,
                                           dim3(256), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

}  // namespace fa
