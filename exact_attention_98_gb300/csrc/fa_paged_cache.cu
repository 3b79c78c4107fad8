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
// Bound by HBM: every row is read once and written once.  A thread takes 16
// elements (a scale's block), the next row's loads in flight while it works on
// one; a block takes 4 tokens, so that looking up their places (page table,
// lengths) is paid once for 4, or 1 where that would leave SMs idle.  Four
// blocks to an SM keep enough loads in flight.  Measured (K, V and Q, d = 128):
// bf16, 13102 tokens of 4 key and 16 query heads: 31.3 us, 5.2 TB/s of 6.7; 4 bits,
// 14631 tokens of 8 and 32 heads, with the rows read back: 96.5 us, 4.1 TB/s.  The
// 4-bit append alone (75 us under a profiler) waits for its loads first (5.4
// cycles per instruction), at 57% of its issue slots, which the divisions by the
// scale, each correctly rounded, and the packing take; four blocks to an SM leave
// it 64 registers, of which 20 spill.  Not kept: 2 or 8 tokens a
// block, a ninth warp that looks the next places up ahead.
#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a block
constexpr int kAppendBlocks = 4;  // blocks of the append on an SM at least

// Eight elements of a row in fp32, as pairs for the packed instructions.
struct Row8 {
  f32x2 x[4];
};

__device__ __forceinline__ Row8 unpack8(const uint4& v) {
  Row8 r;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return r;
}

__device__ __forceinline__ uint4 pack8(const Row8& r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(r.x[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// a c - b s and a c + b s, each product and sum rounded.  The sums are scalar:
// the compiler joins a packed product and a packed sum into one fused operation
// with one rounding.
__device__ __forceinline__ f32x2 turn(f32x2 a, f32x2 b, f32x2 c, f32x2 s) {
  float p0, p1, q0, q1;
  f2_unpack(f2_mul(a, c), p0, p1);
  f2_unpack(f2_mul(b, s), q0, q1);
  return f2_pack(__fsub_rn(p0, q0), __fsub_rn(p1, q1));
}
__device__ __forceinline__ f32x2 turn_back(f32x2 a, f32x2 b, f32x2 c, f32x2 s) {
  float p0, p1, q0, q1;
  f2_unpack(f2_mul(a, c), p0, p1);
  f2_unpack(f2_mul(b, s), q0, q1);
  return f2_pack(__fadd_rn(p0, q0), __fadd_rn(p1, q1));
}

// The largest magnitude, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float amax8(const Row8& r) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(r.x[i], lo, hi);
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(lo)), "f"(fabsf(hi)));
  }
  return m;
}

// Quotients by g rounded to nearest, with r = 1 / g rounded to nearest: the
// quotient's error, exact in one fused operation, corrects it (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  Holds away from overflow and underflow; a negative zero becomes zero.
__device__ __forceinline__ float divide(float x, float g, float r) {
  const float q = __fmul_rn(x, r);
  return fmaf(fmaf(-q, g, x), r, q);
}
__device__ __forceinline__ f32x2 divide(f32x2 x, f32x2 minus_g, f32x2 r) {
  const f32x2 q = f2_mul(x, r);
  return f2_fma(f2_fma(q, minus_g, x), r, q);
}

// The head's factor as the quantisation uses it.
struct Factor {
  float g, r;  // 1 / g rounded to nearest
  bool fits;   // with magnitudes below 2^60, divide() holds
};
__device__ __forceinline__ Factor factor_of(const float* factors, int kvh) {
  Factor f{1.0f, 1.0f, true};
  if (factors) {
    f.g = factors[kvh];
    f.r = __frcp_rn(f.g);
    f.fits = f.g > 0x1p-60f && f.g < 0x1p60f;
  }
  return f;
}

// The scale byte of a block whose largest magnitude is amax: e4m3(amax / g / 6)
// (rounding keeps order, so the largest quotient is the largest magnitude's);
// 0x7F, a NaN, if it is not finite.
__device__ __forceinline__ uint32_t scale_byte(float amax, const Factor& f) {
  constexpr float kSixth = 1.0f / 6.0f;
  float s;
  if (f.fits && amax < 0x1p60f)
    s = divide(divide(amax, f.g, f.r), 6.0f, kSixth);
  else
    s = __fdiv_rn(__fdiv_rn(amax, f.g), 6.0f);
  unsigned short two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(s));
  return s < INFINITY ? two & 0xFFu : 0x7Fu;
}

// 1 / s of an e4m3 scale, rounded to nearest (one Newton step on the hardware's
// approximation; the tests run every scale through it).
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.0f), r, r);
}

// Codes of eight elements x of a block with that scale byte.  y = x / g and z =
// y / s are rounded one by one.  (The order of z and a border between codes is
// that of y and border * s, exact in fp32: two fp32 numbers that differ do so by
// more than a quotient's rounding.)
__device__ __forceinline__ uint32_t codes8(const Row8& x, const Factor& f, bool small, uint32_t byte) {
  if (byte == 0u || byte == 0x7Fu) return 0u;  // zero at this precision, or not finite
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(byte))));
  Row8 y;
  if (small) {
    const f32x2 r2 = f2_pack(f.r, f.r), n2 = f2_pack(-f.g, -f.g);
#pragma unroll
    for (int i = 0; i < 4; ++i) y.x[i] = divide(x.x[i], n2, r2);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_unpack(x.x[i], lo, hi);
      y.x[i] = f2_pack(__fdiv_rn(lo, f.g), __fdiv_rn(hi, f.g));
    }
  }
  const float r = reciprocal(s);
  const f32x2 r2 = f2_pack(r, r), n2 = f2_pack(-s, -s);
  float z[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(divide(y.x[i], n2, r2), z[2 * i], z[2 * i + 1]);
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

// cos and sin of the eight pairs of a thread's chunks, and their rotation.
struct Turn {
  f32x2 cos[4], sin[4];
  int token = -1;  // of the block, whose position they are for

  __device__ __forceinline__ void load(const PagedAppendParams& p, int k, int pos, int2 ch) {
    if (k == token) return;
    token = k;
    const float* at = p.rope + static_cast<size_t>(pos) * p.rot + (p.interleaved ? ch.x * 4 : ch.x * 8);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(at + 4 * u);
      const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(at + (p.rot >> 1) + 4 * u);
      cos[2 * u] = c.x; cos[2 * u + 1] = c.y;
      sin[2 * u] = s.x; sin[2 * u + 1] = s.y;
    }
  }

  __device__ __forceinline__ void apply(Row8& x, Row8& y, bool interleaved) const {
    if (interleaved) {  // four pairs in each chunk
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // two pairs: their first elements together, their second ones together
        Row8& row = u < 2 ? x : y;
        float a0, b0, a1, b1;
        f2_unpack(row.x[2 * (u & 1)], a0, b0);
        f2_unpack(row.x[2 * (u & 1) + 1], a1, b1);
        const f32x2 a = f2_pack(a0, a1), b = f2_pack(b0, b1);
        f2_unpack(turn(a, b, cos[u], sin[u]), a0, a1);
        f2_unpack(turn_back(b, a, cos[u], sin[u]), b0, b1);
        row.x[2 * (u & 1)] = f2_pack(a0, b0);
        row.x[2 * (u & 1) + 1] = f2_pack(a1, b1);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const f32x2 a = x.x[u], b = y.x[u];
        x.x[u] = turn(a, b, cos[u], sin[u]);
        y.x[u] = turn_back(b, a, cos[u], sin[u]);
      }
    }
  }
};

// Records a sequence whose rows do not lie within the tensors' `rows`, or run
// backwards.  By the threads of the first block.  (Not inlined, and ahead of the
// append's first loads: append and read of 14631
// 4-bit tokens 98.9 us inline behind them, 97.1 without the check, 96.5 so.)
__device__ __noinline__ void paged_check_rows(const PagedView& c, const int* cu, int rows,
                                              unsigned int* status) {
  for (int b = threadIdx.x; b < c.B; b += blockDim.x)
    if (cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > rows) record_status(status, kStatusInvalid, kSitePagedRows);
}

// A block of threads takes `tokens` rows of the batch: a thread two chunks of 8
// elements of every 32nd (d = 128) or 64th (d = 64) row of their heads, Q's first,
// then K's and V's, the next row's loads ahead of the present one's work.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int kPer = D / 16;  // threads of a row
  constexpr int kSlots = kThreads / kPer;
  grid_dependency_wait();
  if (blockIdx.x == 0) paged_check_rows(p.c, p.cu, p.rows, p.status);
  __shared__ PagedRow rows[kMaxTokens];
  const int t0 = blockIdx.x * p.tokens;
  const int tokens = min(p.tokens, p.rows - t0);
  const int i = threadIdx.x % kPer;
  const int2 ch = chunk_pair(i, p.rot, p.interleaved);
  const bool turned = ch.x * 8 < p.rot;

  // a thread's elements of the next row of Q (of K or V)
  uint4 next0 = make_uint4(0u, 0u, 0u, 0u), next1 = next0;
  const int q_rows = tokens * p.H;
  auto fetch_q = [&](int r) {
    if (r < q_rows) {
      const int k = p.div_q.div(r), h = r - k * p.H;
      const __nv_bfloat16* src = p.q + static_cast<long long>(t0 + k) * p.q_row + h * p.q_head;
      next0 = *reinterpret_cast<const uint4*>(src + ch.x * 8);
      next1 = *reinterpret_cast<const uint4*>(src + ch.y * 8);
    }
  };
  const int kv_heads = 2 * p.c.Hkv, kv_rows = tokens * kv_heads;
  auto fetch_kv = [&](int r) {
    if (r < kv_rows) {
      const int k = p.div_kv.div(r), h = r - k * kv_heads;
      const __nv_bfloat16* src = h < p.c.Hkv
                                     ? p.k + static_cast<long long>(t0 + k) * p.k_row + h * p.k_head
                                     : p.v + static_cast<long long>(t0 + k) * p.v_row + (h - p.c.Hkv) * p.v_head;
      next0 = *reinterpret_cast<const uint4*>(src + ch.x * 8);
      next1 = *reinterpret_cast<const uint4*>(src + ch.y * 8);
    }
  };
  int r = threadIdx.x / kPer;
  if (q_rows > 0) fetch_q(r);
  else fetch_kv(r);
  if (threadIdx.x < tokens) {
    PagedRow row = paged_row(p.c, p.cu, p.rows, t0 + threadIdx.x, p.status);
    if (row.page >= 0 && p.rot > 0 && row.pos >= p.rope_len) {
      record_status(p.status, kStatusInvalid, kSitePagedLength);
      row.page = -1;
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();

  Turn rope;
  for (; r < q_rows; r += kSlots) {
    Row8 x = unpack8(next0), y = unpack8(next1);
    fetch_q(r + kSlots);
    const int k = p.div_q.div(r);
    if (rows[k].page < 0) continue;
    if (turned) {
      rope.load(p, k, rows[k].pos, ch);
      rope.apply(x, y, p.interleaved);
    }
    __nv_bfloat16* to = p.q_out + (static_cast<long long>(t0) * p.H + r) * D;
    *reinterpret_cast<uint4*>(to + ch.x * 8) = pack8(x);
    *reinterpret_cast<uint4*>(to + ch.y * 8) = pack8(y);
  }

  r = threadIdx.x / kPer;
  if (q_rows > 0) fetch_kv(r);
  const size_t half_bytes = paged_half_bytes(FP4, 1 << p.c.page_shift, D);
  // 4 bits: the other eight elements of each chunk's block of 16 are with these
  // threads of the row
  const int own0 = chunk_owner(ch.x ^ 1, p.rot, p.interleaved), own1 = chunk_owner(ch.y ^ 1, p.rot, p.interleaved);
  const int lane0 = (lane_id() & ~(kPer - 1)) + (own0 >> 1), lane1 = (lane_id() & ~(kPer - 1)) + (own1 >> 1);
  // a warp's rows run together (the shuffles below): all its lanes take part
  // until the last of its rows
  for (int r_warp = (threadIdx.x & ~31) / kPer; r_warp < kv_rows; r_warp += kSlots, r += kSlots) {
    Row8 x = unpack8(next0), y = unpack8(next1);
    fetch_kv(r + kSlots);
    const bool live = r < kv_rows;
    const int k = live ? p.div_kv.div(r) : 0, h = r - k * kv_heads;
    const PagedRow row = rows[k];
    const bool use = live && row.page >= 0;
    const bool is_k = h < p.c.Hkv;
    const int kvh = is_k ? h : h - p.c.Hkv;
    if (use && is_k && turned) {
      rope.load(p, k, row.pos, ch);
      rope.apply(x, y, p.interleaved);
    }
    uint8_t* to = p.c.pages + (static_cast<size_t>(use ? row.page : 0) * p.c.Hkv + kvh) * 2 * half_bytes +
                  (is_k ? 0 : half_bytes);
    if constexpr (FP4) {
      const float m0 = amax8(x), m1 = amax8(y);
      const float a0 = __shfl_sync(0xffffffffu, m0, lane0), a1 = __shfl_sync(0xffffffffu, m1, lane0);
      const float b0 = __shfl_sync(0xffffffffu, m0, lane1), b1 = __shfl_sync(0xffffffffu, m1, lane1);
      const float block0 = max_abs(m0, own0 & 1 ? a1 : a0), block1 = max_abs(m1, own1 & 1 ? b1 : b0);
      if (!use) continue;
      const Factor f = factor_of(is_k ? p.c.k_scale : p.c.v_scale, kvh);
      const uint32_t byte0 = scale_byte(block0, f), byte1 = scale_byte(block1, f);
      const bool small = f.fits && fmaxf(block0, block1) < 0x1p60f;
      uint8_t* codes = to + static_cast<size_t>(row.offset) * (D / 2);
      uint8_t* scales = to + (static_cast<size_t>(D / 2) << p.c.page_shift) + row.offset * (D / 16);
      *reinterpret_cast<uint32_t*>(codes + ch.x * 4) = codes8(x, f, small, byte0);
      *reinterpret_cast<uint32_t*>(codes + ch.y * 4) = codes8(y, f, small, byte1);
      if ((ch.x & 1) == 0) scales[ch.x >> 1] = static_cast<uint8_t>(byte0);
      if ((ch.y & 1) == 0) scales[ch.y >> 1] = static_cast<uint8_t>(byte1);
    } else if (use) {
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
    if (t < p.rows) r = paged_row(p.c, p.cu, p.rows, t, p.status);
    rows[threadIdx.x] = r;
    owned[threadIdx.x] = t < p.rows && t >= p.cu[0] && t < p.cu[p.c.B];
  }
  __syncthreads();
  if (blockIdx.x == 0) paged_check_rows(p.c, p.cu, p.rows, p.status);
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

// One token per block where more would leave multiprocessors idle, four from two
// blocks of four to each of them on.  Append of bf16 (4 bits), one token a block
// against four: 608 rows 8 us against 10 (12 against 14), 1216 rows 12 against 10 (16,
// 16), 2432 rows 17 against 12 (25 against 21), 13000 rows 57 against 38 (88 against 70).
// Read: even up to 608 rows, then 10 against 8, 12 against 8 (12 against 10), 32 against 18.
int tokens_per_block(int rows) { return rows >= sm_count() * 2 * kMaxTokens ? kMaxTokens : 1; }

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
