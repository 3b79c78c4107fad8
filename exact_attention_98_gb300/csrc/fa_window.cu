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
// m16n8k16 mma.sync, whose operands never leave registers:
//   S = Q K_s^T, dP = dO V_s^T, P = exp2(c S - LSE log2 e), dS = P (dP - D),
//   dQ = dS K_s, dK_s += dS^T Q, dV_s += P^T dO
// (dS without the softmax scale, as in the main kernel).  dS and the P of the dV
// product are rounded to bf16, as there.  The lanes of a quad take d in
// runs of D/4, so that Q, dO and O are read 16 bytes at a time.
//
// A key head's queries are cut into parts, each with dK_s and dV_s of its own;
// fa_window_join adds the parts and the main kernel's rows in a fixed order, so
// dK and dV have the same bits from run to run.
#include "fa_device.cuh"
#include "fa_kernels.h"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;  // keys of a pass

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8x8 block of 16-bit values (lane (g, c): row g, columns 2c, 2c + 1) transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// grid slots * BHkv.  A warp takes 16 rows of one query head at a time; lane
// (g, c) their rows g and g + 8, and of each the elements [c D/4, (c+1) D/4).
template <int D>
__global__ void __launch_bounds__(32 * kWarps) fa_window_pre_kernel(const WindowParams p) {
  constexpr int kSteps = D / 16;
  constexpr int kPitch = D + 8;  // of a key row in shared memory: no bank conflicts
  __shared__ __align__(16) __nv_bfloat16 ks[kKeys * kPitch];
  __shared__ __align__(16) __nv_bfloat16 vs[kKeys * kPitch];
  __shared__ __align__(16) float sum[kWarps][kKeys][D];
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, c = lane & 3;
  const int slot = blockIdx.x % p.slots, bkv = blockIdx.x / p.slots;
  grid_dependency_wait();

  const int row_begin = slot * p.slot_rows;
  const int row_end = min(p.N, row_begin + p.slot_rows);
  for (int kb = 0; kb < p.sink_rows / kKeys; ++kb) {
    const int key0 = kb * kKeys;
    __syncthreads();  // the pass before has read ks, vs and sum
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
    float dk[2 * kSteps][4], dv[2 * kSteps][4];
#pragma unroll
    for (int j = 0; j < 2 * kSteps; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dk[j][e] = dv[j][e] = 0.0f;

    for (int h = 0; h < p.group; ++h) {
      const size_t head_row = (static_cast<size_t>(bkv) * p.group + h) * p.N;
      for (int r0 = row_begin + warp * 16; r0 < row_end; r0 += kWarps * 16) {
        // any pair of these rows with keys of this pass?
        const bool far = min(r0 + 15, p.N - 1) - key0 >= p.window;
        if (kb > 0 && !far) continue;
        uint32_t qa[kSteps][4], da[kSteps][4];
        float dsum[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = r0 + g + 8 * r;
          const bool in = row < p.N;
          const size_t at = (head_row + (in ? row : 0)) * D + c * (D / 4);
          dsum[r] = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (in) y = *reinterpret_cast<const uint4*>(p.dout + at + 8 * i);
            if (in && far) x = *reinterpret_cast<const uint4*>(p.q + at + 8 * i);
            qa[2 * i][r] = x.x; qa[2 * i][2 + r] = x.y; qa[2 * i + 1][r] = x.z; qa[2 * i + 1][2 + r] = x.w;
            da[2 * i][r] = y.x; da[2 * i][2 + r] = y.y; da[2 * i + 1][r] = y.z; da[2 * i + 1][2 + r] = y.w;
            if (kb == 0) {
              uint4 o = make_uint4(0u, 0u, 0u, 0u);
              if (in) o = *reinterpret_cast<const uint4*>(p.o + at + 8 * i);
              const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                dsum[r] = fmaf(bf16_lo(ow[e]), bf16_lo(yw[e]), dsum[r]);
                dsum[r] = fmaf(bf16_hi(ow[e]), bf16_hi(yw[e]), dsum[r]);
              }
            }
          }
          if (kb == 0) {
            dsum[r] += __shfl_xor_sync(0xffffffffu, dsum[r], 1);
            dsum[r] += __shfl_xor_sync(0xffffffffu, dsum[r], 2);
            if (in && c == 0) p.dsum[head_row + row] = dsum[r];
          } else {
            dsum[r] = in ? p.dsum[head_row + row] : 0.0f;  // written by this thread's quad in pass 0
          }
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
        float s[2][4], dp[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = dp[nt][e] = 0.0f;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int at = (nt * 8 + g) * kPitch + c * (D / 4) + 4 * k;
            const uint2 kk = *reinterpret_cast<const uint2*>(ks + at);
            const uint2 vv = *reinterpret_cast<const uint2*>(vs + at);
            mma_bf16(s[nt], qa[k], kk.x, kk.y);
            mma_bf16(dp[nt], da[k], vv.x, vv.y);
          }
        }
        uint32_t pp[2][2], dd[2][2];  // P and dS as bf16 pairs: [nt][row]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = r0 + g + 8 * r;
          const float lse = row < p.N ? p.lse[head_row + row] * p.log2e : 0.0f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
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
        // dQ = dS K_s (d in order)
        {
          const uint32_t a[4] = {dd[0][0], dd[0][1], dd[1][0], dd[1][1]};
          const uint32_t row_s = smem_u32(ks) + ((lane & 15) * kPitch + (lane >> 4) * 8) * 2;
#pragma unroll
          for (int j = 0; j < 2 * kSteps; j += 2) {
            uint32_t b[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                         : "r"(row_s + j * 16)
                         : "memory");
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              if (kb > 0) {
                const float2 y0 = in0 ? *reinterpret_cast<const float2*>(acc[0] + 8 * (j + u)) : make_float2(0.f, 0.f);
                const float2 y1 = in1 ? *reinterpret_cast<const float2*>(acc[1] + 8 * (j + u)) : make_float2(0.f, 0.f);
                x[0] = y0.x; x[1] = y0.y; x[2] = y1.x; x[3] = y1.y;
              }
              mma_bf16(x, a, b[2 * u], b[2 * u + 1]);
              if (in0) *reinterpret_cast<float2*>(acc[0] + 8 * (j + u)) = make_float2(x[0], x[1]);
              if (in1) *reinterpret_cast<float2*>(acc[1] + 8 * (j + u)) = make_float2(x[2], x[3]);
            }
          }
        }
        // dK_s += dS^T Q, dV_s += P^T dO: the n-tile of step k, half u holds
        // d = c' D/4 + 4 k + 2 u + e at its column 2 c' + e
        {
          uint32_t at[4], pt[4];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              at[2 * r + nt] = transpose8x8(dd[nt][r]);
              pt[2 * r + nt] = transpose8x8(pp[nt][r]);
            }
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t q0 = transpose8x8(qa[k][2 * u]), q1 = transpose8x8(qa[k][2 * u + 1]);
              mma_bf16(dk[2 * k + u], at, q0, q1);
              const uint32_t d0 = transpose8x8(da[k][2 * u]), d1 = transpose8x8(da[k][2 * u + 1]);
              mma_bf16(dv[2 * k + u], pt, d0, d1);
            }
        }
      }
    }

    // the four warps' dK_s, then dV_s, added in order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which == 1) __syncthreads();
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float* x = which == 0 ? dk[2 * k + u] : dv[2 * k + u];
            *reinterpret_cast<float2*>(&sum[warp][g + 8 * r][c * (D / 4) + 4 * k + 2 * u]) =
                make_float2(x[2 * r], x[2 * r + 1]);
          }
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

// Rows that come in parts.  Blocks below sinks * 2 * BHkv (when there are parts of
// first tokens): a first token's row of dK (times the softmax scale) or dV;
// the thread groups take every kGroups-th part.  Blocks from there on: 256 / d
// rows of a split item's dK or dV, one per thread group.
template <int D>
__global__ void __launch_bounds__(256) fa_window_join_kernel(const WindowParams p) {
  constexpr int kGroups = 256 / D;
  __shared__ float part[kGroups][D];
  grid_dependency_wait();
  const int col = threadIdx.x % D, grp = threadIdx.x / D;
  const int sink_blocks = p.slots > 0 ? p.sinks * 2 * p.BHkv : 0;
  // element (row, col) of part k of an item, and whether an item is in parts
  auto tile_row = [&](int item, int k, int which, int row) {
    return p.tile_part[((static_cast<size_t>((item - p.split_from) * p.split_parts + k) * 2 + which) * kBlockN + row) * D + col];
  };
  if (static_cast<int>(blockIdx.x) >= sink_blocks) {
    const int rest = static_cast<int>(blockIdx.x) - sink_blocks;
    constexpr int kPerItem = 2 * kBlockN / kGroups;  // blocks of an item
    const int item = p.split_from + rest / kPerItem;
    const int at = rest % kPerItem * kGroups + grp;
    const int which = at / kBlockN, row = at % kBlockN;
    const int bkv = item / p.n_kblk, key = item % p.n_kblk * kBlockN + row;
    if (key >= p.N || (p.slots > 0 && key < p.sinks)) return;
    float x = 0.0f;
#pragma unroll 4
    for (int k = 0; k < p.split_parts; ++k) x += tile_row(item, k, which, row);
    __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N + key) * D + col;
    *out = __float2bfloat16_rn(which == 0 ? x * p.scale : x);
    return;
  }
  const int key = blockIdx.x % p.sinks, which = (blockIdx.x / p.sinks) & 1, bkv = blockIdx.x / p.sinks / 2;
  const size_t stride = static_cast<size_t>(p.BHkv) * 2 * p.sink_rows * D;
  const float* from = p.sink_part + ((static_cast<size_t>(bkv) * 2 + which) * p.sink_rows + key) * D + col;
  const int item = bkv * p.n_kblk;  // its first key tile
  const bool split = item >= p.split_from;
  float x = 0.0f;
#pragma unroll 8
  for (int s = grp; s < p.slots + (split ? 0 : 1); s += kGroups) x += from[s * stride];
  if (split)
    for (int k = grp; k < p.split_parts; k += kGroups) x += tile_row(item, k, which, key);
  part[grp][col] = x;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) x += part[k][col];
  __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<size_t>(bkv) * p.N + key) * D + col;
  *out = __float2bfloat16_rn(which == 0 ? x * p.scale : x);
}

}  // namespace

cudaError_t launch_window_pre(const WindowParams& p, int d, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned int>(p.slots) * static_cast<unsigned int>(p.BHkv));
  const cudaError_t err = launch_dependent(d == 128 ? fa_window_pre_kernel<128> : fa_window_pre_kernel<64>, grid,
                                           dim3(32 * kWarps), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_window_join(const WindowParams& p, int d, cudaStream_t stream) {
  const unsigned int items = static_cast<unsigned int>(p.n_kblk * p.BHkv - p.split_from);
  const dim3 grid((p.slots > 0 ? static_cast<unsigned int>(p.sinks) * 2u * static_cast<unsigned int>(p.BHkv) : 0u) +
                  items * (2u * kBlockN / (256u / static_cast<unsigned int>(d))));
  const cudaError_t err = launch_dependent(d == 128 ? fa_window_join_kernel<128> : fa_window_join_kernel<64>, grid,
                                           dim3(256), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

}  // namespace fa
