// Rotation of Q and K rows by their positions, and its transpose:
//   x'_a = x_a cos - x_b sin,  x'_b = x_b cos + x_a sin
// with cos and sin of pair i at the row's position from an fp32 table; a pair is
// (i, i + rot/2) or (2i, 2i + 1).  The transpose has -sin for sin: what the gradient of
// x' is to be multiplied by.  Products and sums are rounded to fp32 each, as in the
// paged cache's append, so both give the same bits.
//
// HBM bounds it: every element is read and written once, a few operations each.  A
// thread takes 16 elements (8 pairs: two 16-byte loads) of kHeads heads of one row,
// all loads before the first use, and the pairs' cos and sin once for these
// heads.  16384 rows, H = 32, Hkv = 8, d = 128: 51 us, 6.6 TB/s.  Three heads to a
// thread are 64 registers; 1, 2, 4 and 8 heads took 65, 62, 58 and 62 us against 58,
// 4999 rows of 20 heads 17, 17, 17 and 17 against 15 (timed one by one).
#include "fa_packed.cuh"

namespace fa {
namespace {

constexpr int kRotateThreads = 256;

// kHeads heads to a thread; kInterleaved: pairs are neighbours.
template <int D, int kHeads, bool kInterleaved>
__global__ void __launch_bounds__(kRotateThreads) fa_rotate_kernel(const __grid_constant__ RotateParams p) {
  constexpr int kUnits = D / 16;  // of 16 elements, in a row of a head
  grid_dependency_wait();
  const long long i = blockIdx.x * static_cast<long long>(kRotateThreads) + threadIdx.x;
  const int u = static_cast<int>(i % kUnits);
  const uint32_t rest = static_cast<uint32_t>(i / kUnits);
  const int row = static_cast<int>(p.div_chunks.div(rest));
  if (row >= p.rows) return;
  const int head0 = static_cast<int>(rest - static_cast<uint32_t>(row) * p.div_chunks.d) * kHeads;
  const int pos = p.positions[row];
  if (pos < 0) return;  // a row of no sequence
  if (pos >= p.rope_len) {
    if (u == 0) record_status(p.status, kPackedInvalid, kSitePackedPosition);
    return;
  }
  // the unit's two runs of 8 elements
  const bool turned = u * 16 < p.rot;
  const int e0 = kInterleaved || !turned ? u * 16 : u * 8;
  const int e1 = kInterleaved || !turned ? u * 16 + 8 : u * 8 + p.rot / 2;
  uint4 x[kHeads], y[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int head = head0 + h;
    if (head < p.H + p.Hkv) {
      const __nv_bfloat16* src = head < p.H ? p.q + row * p.q_row + head * p.q_head
                                            : p.k + row * p.k_row + (head - p.H) * p.k_head;
      x[h] = *reinterpret_cast<const uint4*>(src + e0);
      y[h] = *reinterpret_cast<const uint4*>(src + e1);
    }
  }
  float cs[8], sn[8];
  if (turned) {
    const float* t = p.rope + static_cast<size_t>(pos) * p.rot + u * 8;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float4 a = *reinterpret_cast<const float4*>(t + 4 * c);
      const float4 b = *reinterpret_cast<const float4*>(t + p.rot / 2 + 4 * c);
      cs[4 * c] = a.x; cs[4 * c + 1] = a.y; cs[4 * c + 2] = a.z; cs[4 * c + 3] = a.w;
      sn[4 * c] = b.x; sn[4 * c + 1] = b.y; sn[4 * c + 2] = b.z; sn[4 * c + 3] = b.w;
    }
    if (p.backward) {
#pragma unroll
      for (int c = 0; c < 8; ++c) sn[c] = -sn[c];
    }
  }
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  auto turn = [](float a, float b, float c, float s, float& a1, float& b1) {
    a1 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b1 = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  };
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int head = head0 + h;
    if (head >= p.H + p.Hkv) break;
    uint32_t xw[4] = {x[h].x, x[h].y, x[h].z, x[h].w}, yw[4] = {y[h].x, y[h].y, y[h].z, y[h].w};
    if (turned) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a0, a1, b0, b1;
        if constexpr (kInterleaved) {  // a word is a pair
          turn(lo(xw[c]), hi(xw[c]), cs[c], sn[c], a0, a1);
          turn(lo(yw[c]), hi(yw[c]), cs[4 + c], sn[4 + c], b0, b1);
        } else {
          turn(lo(xw[c]), lo(yw[c]), cs[2 * c], sn[2 * c], a0, b0);
          turn(hi(xw[c]), hi(yw[c]), cs[2 * c + 1], sn[2 * c + 1], a1, b1);
        }
        xw[c] = pack_bf16x2(a0, a1);
        yw[c] = pack_bf16x2(b0, b1);
      }
    }
    __nv_bfloat16* dst = head < p.H ? p.q_out + row * p.qo_row + head * p.qo_head
                                    : p.k_out + row * p.ko_row + (head - p.H) * p.ko_head;
    *reinterpret_cast<uint4*>(dst + e0) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
    *reinterpret_cast<uint4*>(dst + e1) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
  }
}

template <int D, int kHeads>
cudaError_t launch(RotateParams& p, cudaStream_t stream) {
  const int chunks = (p.H + p.Hkv + kHeads - 1) / kHeads;
  p.div_chunks = FastDiv(static_cast<uint32_t>(chunks));
  const long long threads = static_cast<long long>(p.rows) * chunks * (D / 16);
  const long long blocks = (threads + kRotateThreads - 1) / kRotateThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t err = launch_dependent(
      p.interleaved ? fa_rotate_kernel<D, kHeads, true> : fa_rotate_kernel<D, kHeads, false>,
      dim3(static_cast<unsigned int>(blocks)), dim3(kRotateThreads), 0, stream, p);
  return err != cudaSuccess ? err : launched(1);
}

}  // namespace

cudaError_t launch_rotate(RotateParams p, int d, cudaStream_t stream) {
  if (d == 128) return launch<128, 3>(p, stream);
  if (d == 64) return launch<64, 3>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
