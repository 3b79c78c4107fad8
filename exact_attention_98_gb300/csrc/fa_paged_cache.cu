// The paged key/value cache: appending rotated rows, and reading rows back.
//
// Append: row x of K (and of Q) at position p is rotated in pairs,
//   x'_a = x_a cos - x_b sin,  x'_b = x_b cos + x_a sin,
// with cos and sin of pair i at p from an fp32 table; a pair is (i, i + rot/2)
// or, interleaved, (2i, 2i+1); elements from rot on stay.  Products and their
// sum are rounded to fp32 one by one, so that a plain fp32 evaluation gives
// the same bits, which a 4-bit code at the border of two needs.  The result
// is rounded once: to bf16, or to 4 bits: with g the head's factor and the
// block of 16's y = x' / g, s = e4m3(max|y| / 6) and code = e2m1(y / s), each
// rounded to nearest, ties to even.  A block that holds an infinity or a NaN
// gets the scale NaN: it reads back as NaN.
//
// Bound by HBM: every row is read once and written once.
#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a block

struct Row8 {
  float x[8];
};

__device__ __forceinline__ Row8 unpack8(const uint4& v) {
  Row8 r;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

__device__ __forceinline__ uint4 pack8(const Row8& r) {
  return make_uint4(pack_bf16x2(r.x[0], r.x[1]), pack_bf16x2(r.x[2], r.x[3]),
                    pack_bf16x2(r.x[4], r.x[5]), pack_bf16x2(r.x[6], r.x[7]));
}

__device__ __forceinline__ float turn(float a, float b, float cos, float sin) {
  return __fsub_rn(__fmul_rn(a, cos), __fmul_rn(b, sin));
}
__device__ __forceinline__ float turn_back(float a, float b, float cos, float sin) {
  return __fadd_rn(__fmul_rn(a, cos), __fmul_rn(b, sin));
}

// x / g rounded to nearest with r = 1 / g rounded to nearest: the quotient's
// error, exact in one fused operation, corrects it (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  Holds
// away from overflow and underflow; the sign of a zero is x's.
__device__ __forceinline__ float divide(float x, float g, float r) {
  const float q = __fmul_rn(x, r);
  return copysignf(fmaf(fmaf(-q, g, x), r, q), x);
}

// Eight of a block's 16 elements over the head's factor, their largest magnitude
// (NaN where one is not finite).
__device__ __forceinline__ float scale8(Row8& x, float g) {
  float amax = 0.0f, zero = 0.0f;
  if (g != 1.0f) {
    const float r = __frcp_rn(g);
    const bool fast = g > 0x1p-60f && g < 0x1p60f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.x[i] = fast && fabsf(x.x[i]) < 0x1p60f ? divide(x.x[i], g, r) : __fdiv_rn(x.x[i], g);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(x.x[i]));
    zero = fmaf(x.x[i], 0.0f, zero);
  }
  return amax + zero;
}

// The block's scale byte from its largest magnitude (NaN: 0x7F), and its codes.
// An element's quotient by the scale has to be on the right side of the borders
// between codes: these times the scale are exact in fp32, and two fp32 numbers
// that differ do so by more than a quotient's rounding, so the rounded quotient
// is on the exact one's side.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float s = __fdiv_rn(amax, 6.0f);
  unsigned short two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(s));
  return amax == amax ? two & 0xFFu : 0x7Fu;
}
__device__ __forceinline__ uint32_t codes8(const Row8& y, uint32_t byte) {
  if (byte == 0u || byte == 0x7Fu) return 0u;  // zero at this precision, or not finite
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(byte))));
  const float r = __frcp_rn(s);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = divide(y.x[i], s, r);
  uint32_t codes;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(codes)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  return codes;
}

// Which two chunks of 8 elements thread i of a row's D/16 takes: both ends of 8
// pairs (i, i + rot/2); behind the rotated part, and interleaved, neighbours.
__device__ __forceinline__ int2 chunk_pair(int i, int rot, bool interleaved) {
  const int half8 = rot >> 4;  // chunks of half the rotated part
  if (interleaved) return make_int2(2 * i, 2 * i + 1);
  if (i < half8) return make_int2(i, i + half8);
  return make_int2(2 * i, 2 * i + 1);
}
// The thread that takes chunk x, times 2, plus 1 if as its second one.
__device__ __forceinline__ int chunk_owner(int x, int rot, bool interleaved) {
  const int half8 = rot >> 4;
  if (interleaved || x >= 2 * half8) return x;
  return x < half8 ? 2 * x : 2 * (x - half8) + 1;
}

// A block of threads takes `tokens` rows of the batch; a thread two chunks of 8
// elements of every 32nd (d = 128) or 64th (d = 64) of their heads' rows (Q heads,
// then K heads, then V heads, token by token), the next row's loads ahead of
// the present one's work.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int kPer = D / 16;  // threads of a row
  constexpr int kSlots = kThreads / kPer;
  grid_dependency_wait();
  __shared__ PagedRow rows[kMaxTokens];
  const int t0 = blockIdx.x * p.tokens;
  const int hq = p.H;  // 0 without Q
  const int heads = static_cast<int>(p.div_heads.d);
  const int i = threadIdx.x % kPer;
  const int2 ch = chunk_pair(i, p.rot, p.interleaved);
  const int n_rows = min(p.tokens, p.rows - t0) * heads;
  auto source = [&](int r) {
    const int k = p.div_heads.div(r), h = r - k * heads;
    const long long t = t0 + k;
    return h < hq                ? p.q + t * p.q_row + h * p.q_head
           : h < hq + p.c.Hkv    ? p.k + t * p.k_row + (h - hq) * p.k_head
                                 : p.v + t * p.v_row + (h - hq - p.c.Hkv) * p.v_head;
  };
  uint4 next0 = make_uint4(0u, 0u, 0u, 0u), next1 = next0;
  auto fetch = [&](int r) {
    if (r < n_rows) {
      const __nv_bfloat16* src = source(r);
      next0 = *reinterpret_cast<const uint4*>(src + ch.x * 8);
      next1 = *reinterpret_cast<const uint4*>(src + ch.y * 8);
    }
  };
  int r = threadIdx.x / kPer;
  fetch(r);
  if (threadIdx.x < p.tokens) {
    const int t = t0 + threadIdx.x;
    PagedRow row{-1, 0, -1};
    if (t < p.rows) row = paged_row(p.c, p.cu, t, p.status);
    if (row.page >= 0 && p.rot > 0 && row.pos >= p.rope_len) {
      record_status(p.status, kStatusInvalid, kSitePagedLength);
      row.page = -1;
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
  const int half = p.rot >> 1;
  const size_t half_bytes = paged_half_bytes(FP4, 1 << p.c.page_shift, D);
  // 4 bits: the other eight elements of each chunk's block of 16 are with these
  // threads of the row
  const int own0 = chunk_owner(ch.x ^ 1, p.rot, p.interleaved), own1 = chunk_owner(ch.y ^ 1, p.rot, p.interleaved);
  const int lane0 = (lane_id() & ~(kPer - 1)) + (own0 >> 1), lane1 = (lane_id() & ~(kPer - 1)) + (own1 >> 1);
  int at_token = -1;
  float cos[8], sin[8];
  // a warp's rows run together (the shuffles below): all its lanes take part
  // until the last of its rows
  for (int r_warp = (threadIdx.x & ~31) / kPer; r_warp < n_rows; r_warp += kSlots, r += kSlots) {
    const bool live = r < n_rows;
    Row8 x = unpack8(next0), y = unpack8(next1);
    fetch(r + kSlots);
    const int k = live ? p.div_heads.div(r) : 0, h = r - k * heads;
    const PagedRow row = rows[k];
    const bool is_q = h < hq;
    const bool is_k = !is_q && h < hq + p.c.Hkv;
    const int kvh = is_q ? 0 : (h - hq) - (is_k ? 0 : p.c.Hkv);
    const bool use = live && row.page >= 0;
    if (use && (is_q || is_k) && ch.x * 8 < p.rot) {
      if (k != at_token) {
        at_token = k;
        const float* at = p.rope + static_cast<size_t>(row.pos) * p.rot + (p.interleaved ? ch.x * 4 : ch.x * 8);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float4 c = *reinterpret_cast<const float4*>(at + 4 * u);
          const float4 s = *reinterpret_cast<const float4*>(at + half + 4 * u);
          cos[4 * u] = c.x; cos[4 * u + 1] = c.y; cos[4 * u + 2] = c.z; cos[4 * u + 3] = c.w;
          sin[4 * u] = s.x; sin[4 * u + 1] = s.y; sin[4 * u + 2] = s.z; sin[4 * u + 3] = s.w;
        }
      }
      if (p.interleaved) {  // pairs 8 i .. 8 i + 7: four in each chunk
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float a = x.x[2 * u], b = x.x[2 * u + 1], e = y.x[2 * u], f = y.x[2 * u + 1];
          x.x[2 * u] = turn(a, b, cos[u], sin[u]);
          x.x[2 * u + 1] = turn_back(b, a, cos[u], sin[u]);
          y.x[2 * u] = turn(e, f, cos[4 + u], sin[4 + u]);
          y.x[2 * u + 1] = turn_back(f, e, cos[4 + u], sin[4 + u]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float a = x.x[u], b = y.x[u];
          x.x[u] = turn(a, b, cos[u], sin[u]);
          y.x[u] = turn_back(b, a, cos[u], sin[u]);
        }
      }
    }
    if (use && is_q) {
      __nv_bfloat16* to = p.q_out + ((static_cast<long long>(t0) + k) * p.H + h) * D;
      *reinterpret_cast<uint4*>(to + ch.x * 8) = pack8(x);
      *reinterpret_cast<uint4*>(to + ch.y * 8) = pack8(y);
    }
    uint8_t* to = p.c.pages + (static_cast<size_t>(use ? row.page : 0) * p.c.Hkv + kvh) * 2 * half_bytes +
                  (is_k ? 0 : half_bytes);
    if constexpr (FP4) {
      const float* factor = is_k ? p.c.k_scale : p.c.v_scale;
      const bool cached = use && !is_q;
      const float g = cached && factor ? factor[kvh] : 1.0f;
      if (__any_sync(0xffffffffu, cached)) {
        const float m0 = scale8(x, g), m1 = scale8(y, g);
        const float a0 = __shfl_sync(0xffffffffu, m0, lane0), a1 = __shfl_sync(0xffffffffu, m1, lane0);
        const float b0 = __shfl_sync(0xffffffffu, m0, lane1), b1 = __shfl_sync(0xffffffffu, m1, lane1);
        const float o0 = own0 & 1 ? a1 : a0, o1 = own1 & 1 ? b1 : b0;
        // (0 times each added: NaN where either is)
        const uint32_t byte0 = scale_byte(fmaxf(m0, o0) + fmaf(m0, 0.0f, o0 * 0.0f));
        const uint32_t byte1 = scale_byte(fmaxf(m1, o1) + fmaf(m1, 0.0f, o1 * 0.0f));
        if (cached) {
          uint8_t* codes = to + static_cast<size_t>(row.offset) * (D / 2);
          uint8_t* scales = to + (static_cast<size_t>(D / 2) << p.c.page_shift) + row.offset * (D / 16);
          *reinterpret_cast<uint32_t*>(codes + ch.x * 4) = codes8(x, byte0);
          *reinterpret_cast<uint32_t*>(codes + ch.y * 4) = codes8(y, byte1);
          if ((ch.x & 1) == 0) scales[ch.x >> 1] = static_cast<uint8_t>(byte0);
          if ((ch.y & 1) == 0) scales[ch.y >> 1] = static_cast<uint8_t>(byte1);
        }
      }
    } else if (use && !is_q) {
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(to) + static_cast<size_t>(row.offset) * D;
      *reinterpret_cast<uint4*>(out + ch.x * 8) = pack8(x);
      *reinterpret_cast<uint4*>(out + ch.y * 8) = pack8(y);
    }
  }
}

// The same rows out of the cache as bf16 [rows, Hkv, d]; a row without a usable
// place reads as zeros, rows behind the last sequence are left alone.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  constexpr int kPer = D / 16;  // threads of a row
  constexpr int kSlots = kThreads / kPer;
  grid_dependency_wait();
  __shared__ PagedRow rows[kMaxTokens];
  __shared__ int owned[kMaxTokens];
  const int t0 = blockIdx.x * p.tokens;
  if (threadIdx.x < p.tokens) {
    const int t = t0 + threadIdx.x;
    PagedRow r{-1, 0, -1};
    if (t < p.rows) r = paged_row(p.c, p.cu, t, p.status);
    rows[threadIdx.x] = r;
    owned[threadIdx.x] = t < p.rows && t >= p.cu[0] && t < p.cu[p.c.B];
  }
  __syncthreads();
  const int i = threadIdx.x % kPer;
  const size_t half_bytes = paged_half_bytes(FP4, 1 << p.c.page_shift, D);
  const int heads = 2 * p.c.Hkv;  // K heads, then V heads
  const int n_rows = min(p.tokens, p.rows - t0) * heads;
  // 16 elements of a row per thread, four rows' loads ahead of their stores
  constexpr int kBatch = 4;
  for (int r0 = threadIdx.x / kPer; r0 < n_rows; r0 += kBatch * kSlots) {
    uint4 a[kBatch], b[kBatch];  // bf16: the elements; 4 bits: a.x, a.y codes, a.z scale byte
    float mul[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      mul[u] = 1.0f;
      const int r = r0 + u * kSlots;
      if (r >= n_rows) continue;
      const int k = p.div_heads.div(r), h = r - k * heads;
      const PagedRow row = rows[k];
      if (row.page < 0) continue;
      const bool is_k = h < p.c.Hkv;
      const int kvh = is_k ? h : h - p.c.Hkv;
      const uint8_t* from = p.c.pages + (static_cast<size_t>(row.page) * p.c.Hkv + kvh) * 2 * half_bytes +
                            (is_k ? 0 : half_bytes);
      if constexpr (FP4) {
        const float* g = is_k ? p.c.k_scale : p.c.v_scale;
        if (g) mul[u] = g[kvh];
        const uint2 codes = *reinterpret_cast<const uint2*>(from + static_cast<size_t>(row.offset) * (D / 2) + i * 8);
        a[u].x = codes.x;
        a[u].y = codes.y;
        a[u].z = from[(static_cast<size_t>(D / 2) << p.c.page_shift) + row.offset * (D / 16) + i];
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(from + (static_cast<size_t>(row.offset) * D + i * 16) * 2);
        a[u] = src[0];
        b[u] = src[1];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = r0 + u * kSlots;
      if (r >= n_rows) break;
      const int k = p.div_heads.div(r), h = r - k * heads;
      if (!owned[k]) continue;
      if constexpr (FP4) {
        const uint32_t s2 = e4m3x2_to_f16x2(a[u].z * 0x101u);
        const uint32_t codes[2] = {a[u].x, a[u].y};
        uint32_t out[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[4];
          e2m1x8_to_f16x2(codes[c], w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t v2 = hmul2(w[e], s2);  // exact: six bits at most
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v2));
            out[4 * c + e] = pack_bf16x2(f.x * mul[u], f.y * mul[u]);
          }
        }
        a[u] = make_uint4(out[0], out[1], out[2], out[3]);
        b[u] = make_uint4(out[4], out[5], out[6], out[7]);
      }
      const bool is_k = h < p.c.Hkv;
      const int kvh = is_k ? h : h - p.c.Hkv;
      uint4* to = reinterpret_cast<uint4*>(
          (is_k ? p.k : p.v) + ((static_cast<long long>(t0) + k) * p.c.Hkv + kvh) * D + i * 16);
      to[0] = a[u];
      to[1] = b[u];
    }
  }
}

// One token per block while that leaves multiprocessors idle otherwise.
int tokens_per_block(int rows) { return rows >= 152 * 8 * kMaxTokens ? kMaxTokens : 1; }

}  // namespace

cudaError_t launch_paged_append(PagedAppendParams p, int d, bool fp4, cudaStream_t stream) {
  p.tokens = tokens_per_block(p.rows);
  const dim3 grid(static_cast<unsigned int>((p.rows + p.tokens - 1) / p.tokens));
  auto kernel = d == 128 ? (fp4 ? paged_append_kernel<128, true> : paged_append_kernel<128, false>)
                         : (fp4 ? paged_append_kernel<64, true> : paged_append_kernel<64, false>);
  const cudaError_t err = launch_dependent(kernel, grid, dim3(kThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

cudaError_t launch_paged_read(PagedReadParams p, int d, bool fp4, cudaStream_t stream) {
  p.tokens = tokens_per_block(p.rows);
  const dim3 grid(static_cast<unsigned int>((p.rows + p.tokens - 1) / p.tokens));
  auto kernel = d == 128 ? (fp4 ? paged_read_kernel<128, true> : paged_read_kernel<128, false>)
                         : (fp4 ? paged_read_kernel<64, true> : paged_read_kernel<64, false>);
  const cudaError_t err = launch_dependent(kernel, grid, dim3(kThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

}  // namespace fa
