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

// Eight of a block's 16 elements (the other eight in the neighbouring lane)
// -> their codes in one word, and the block's scale byte.
__device__ __forceinline__ uint32_t quantise8(const Row8& r, float g, uint32_t& scale_byte) {
  float y[8], amax = 0.0f, zero = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = __fdiv_rn(r.x[i], g);
    amax = fmaxf(amax, fabsf(y[i]));
    zero += y[i] * 0.0f;  // NaN if y is not finite
  }
  const unsigned int pair = 3u << (lane_id() & ~1);
  amax = fmaxf(amax, __shfl_xor_sync(pair, amax, 1));
  zero += __shfl_xor_sync(pair, zero, 1);
  if (!(zero == 0.0f)) {
    scale_byte = 0x7Fu;
    return 0u;
  }
  float s = __fdiv_rn(amax, 6.0f);
  unsigned short two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(s));
  scale_byte = two & 0xFFu;
  if (scale_byte == 0u) return 0u;  // the block is zero at this precision
  s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(scale_byte))));
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = __fdiv_rn(y[i], s);
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

// A block of threads takes `tokens` rows of the batch; a thread one chunk of
// 8 elements, of every 16th (d = 128) or 32nd (d = 64) head's row: Q heads,
// then K heads, then V heads.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedAppendParams p) {
  constexpr int kChunks = D / 8;
  constexpr int kSlots = kThreads / kChunks;
  grid_dependency_wait();
  __shared__ PagedRow rows[kMaxTokens];
  const int t0 = blockIdx.x * p.tokens;
  if (threadIdx.x < p.tokens) {
    const int t = t0 + threadIdx.x;
    PagedRow r{-1, 0, -1};
    if (t < p.rows) r = paged_row(p.c, p.cu, t, p.status);
    if (r.page >= 0 && p.rot > 0 && r.pos >= p.rope_len) {
      record_status(p.status, kStatusInvalid, kSitePagedLength);
      r.page = -1;
    }
    rows[threadIdx.x] = r;
  }
  __syncthreads();
  const int chunk = threadIdx.x % kChunks;
  const int slot = threadIdx.x / kChunks;
  const int e0 = chunk * 8;
  const int half = p.rot >> 1;
  const bool turned = e0 < p.rot;
  const bool low = e0 < half;  // this chunk holds the pairs' first elements
  const int hq = p.q ? p.H : 0;
  const int heads = hq + 2 * p.c.Hkv;
  const size_t half_bytes = paged_half_bytes(FP4, 1 << p.c.page_shift, D);
  for (int k = 0; k < p.tokens; ++k) {
    const PagedRow r = rows[k];
    if (r.page < 0) continue;
    const long long t = t0 + k;
    float cos[8], sin[8];
    if (turned) {
      const float* at = p.rope + static_cast<size_t>(r.pos) * p.rot;
      if (p.interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(at + chunk * 4);
        const float4 s = *reinterpret_cast<const float4*>(at + half + chunk * 4);
        cos[0] = c.x; cos[1] = c.y; cos[2] = c.z; cos[3] = c.w;
        sin[0] = s.x; sin[1] = s.y; sin[2] = s.z; sin[3] = s.w;
      } else {
        const int i0 = low ? e0 : e0 - half;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 c = *reinterpret_cast<const float4*>(at + i0 + 4 * i);
          const float4 s = *reinterpret_cast<const float4*>(at + half + i0 + 4 * i);
          cos[4 * i] = c.x; cos[4 * i + 1] = c.y; cos[4 * i + 2] = c.z; cos[4 * i + 3] = c.w;
          sin[4 * i] = s.x; sin[4 * i + 1] = s.y; sin[4 * i + 2] = s.z; sin[4 * i + 3] = s.w;
        }
      }
    }
    for (int h = slot; h < heads; h += kSlots) {
      const bool is_q = h < hq;
      const bool is_k = !is_q && h < hq + p.c.Hkv;
      const int kvh = is_q ? 0 : (h - hq) - (is_k ? 0 : p.c.Hkv);
      const __nv_bfloat16* src =
          is_q   ? p.q + t * p.q_row + h * p.q_head
          : is_k ? p.k + t * p.k_row + kvh * p.k_head
                 : p.v + t * p.v_row + kvh * p.v_head;
      const uint4 own = *reinterpret_cast<const uint4*>(src + e0);
      Row8 x = unpack8(own);
      if (turned && (is_q || is_k)) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x.x[2 * i], b = x.x[2 * i + 1];
            x.x[2 * i] = turn(a, b, cos[i], sin[i]);
            x.x[2 * i + 1] = turn_back(b, a, cos[i], sin[i]);
          }
        } else {
          const Row8 o = unpack8(*reinterpret_cast<const uint4*>(src + (low ? e0 + half : e0 - half)));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x.x[i] = low ? turn(x.x[i], o.x[i], cos[i], sin[i])
                         : turn_back(x.x[i], o.x[i], cos[i], sin[i]);
        }
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + (t * p.H + h) * D + e0) = pack8(x);
        continue;
      }
      uint8_t* to = p.c.pages + (static_cast<size_t>(r.page) * p.c.Hkv + kvh) * 2 * half_bytes +
                    (is_k ? 0 : half_bytes);
      if constexpr (FP4) {
        const float* g = is_k ? p.c.k_scale : p.c.v_scale;
        uint32_t scale;
        const uint32_t codes = quantise8(x, g ? g[kvh] : 1.0f, scale);
        *reinterpret_cast<uint32_t*>(to + static_cast<size_t>(r.offset) * (D / 2) + chunk * 4) = codes;
        if ((chunk & 1) == 0)
          to[(static_cast<size_t>(D / 2) << p.c.page_shift) + r.offset * (D / 16) + (chunk >> 1)] =
              static_cast<uint8_t>(scale);
      } else {
        *reinterpret_cast<uint4*>(to + (static_cast<size_t>(r.offset) * D + e0) * 2) = pack8(x);
      }
    }
  }
}

// The same rows out of the cache as bf16 [rows, Hkv, d]; a row without a usable
// place reads as zeros, rows behind the last sequence are left alone.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const PagedReadParams p) {
  constexpr int kChunks = D / 8;
  constexpr int kSlots = kThreads / kChunks;
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
  const int chunk = threadIdx.x % kChunks;
  const int slot = threadIdx.x / kChunks;
  const size_t half_bytes = paged_half_bytes(FP4, 1 << p.c.page_shift, D);
  for (int k = 0; k < p.tokens; ++k) {
    if (!owned[k]) continue;
    const PagedRow r = rows[k];
    const long long t = t0 + k;
    for (int h = slot; h < 2 * p.c.Hkv; h += kSlots) {
      const bool is_k = h < p.c.Hkv;
      const int kvh = is_k ? h : h - p.c.Hkv;
      uint4 out = make_uint4(0u, 0u, 0u, 0u);
      if (r.page >= 0) {
        const uint8_t* from = p.c.pages +
                              (static_cast<size_t>(r.page) * p.c.Hkv + kvh) * 2 * half_bytes +
                              (is_k ? 0 : half_bytes);
        if constexpr (FP4) {
          const float* g = is_k ? p.c.k_scale : p.c.v_scale;
          const float mul = g ? g[kvh] : 1.0f;
          const uint32_t codes = *reinterpret_cast<const uint32_t*>(
              from + static_cast<size_t>(r.offset) * (D / 2) + chunk * 4);
          const uint32_t scale =
              from[(static_cast<size_t>(D / 2) << p.c.page_shift) + r.offset * (D / 16) + (chunk >> 1)];
          const uint32_t s2 = e4m3x2_to_f16x2(scale | (scale << 8));
          uint32_t w[4], o[4];
          e2m1x8_to_f16x2(codes, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v2 = hmul2(w[i], s2);  // exact: six bits at most
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v2));
            o[i] = pack_bf16x2(f.x * mul, f.y * mul);
          }
          out = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          out = *reinterpret_cast<const uint4*>(from + (static_cast<size_t>(r.offset) * D + chunk * 8) * 2);
        }
      }
      __nv_bfloat16* to = (is_k ? p.k : p.v) + (t * p.c.Hkv + kvh) * D + chunk * 8;
      *reinterpret_cast<uint4*>(to) = out;
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
