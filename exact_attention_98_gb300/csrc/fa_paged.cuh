// Shared by the kernels of the paged key/value cache: its layout, which row of
// a ragged batch belongs to which sequence, and the 4-bit format.
//
// A block is what one page holds for one key head: the K rows of the page's
// page_size positions, then the V rows.  bf16: rows of d values.  4 bits: the
// rows' codes (d/2 bytes each, e2m1, even element in the low nibble), then
// their scales (d/16 bytes each, e4m3, one per 16 consecutive elements);
// value = code * scale * (the head's factor).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_device.cuh"
#include "fa_kernels.h"

namespace fa {

// Site codes recorded with FA_ERR_INVALID_ARG (1) when the batch's own tables
// are not usable.
constexpr unsigned int kStatusInvalid = 1u;
enum : unsigned int {
  kSitePagedRows = 0x501,    // cu_new does not fit the rows, or more rows than max_new
  kSitePagedLength = 0x502,  // a sequence longer than its pages, or its rotation table
  kSitePagedPage = 0x503,    // a page number outside the cache
};

// Bytes of a block's K half (its V half has as many).
__host__ __device__ constexpr size_t paged_half_bytes(bool fp4, int page_size, int d) {
  return static_cast<size_t>(page_size) * (fp4 ? d / 2 + d / 16 : 2 * d);
}

// Where a new row goes: sequence, position, and its place in the cache.
struct PagedRow {
  int page;    // page number, -1: no place (padding, or a bad table: recorded)
  int offset;  // position within the page
  int pos;     // position within the sequence
};

// Row t belongs to the sequence b with cu[b] <= t < cu[b+1] and holds its
// position seq_lens[b] - cu[b+1] + t (the rows are the sequence's last).
__device__ __forceinline__ PagedRow paged_row(const PagedView& c, const int* cu, int rows, int t,
                                              unsigned int* status) {
  PagedRow r{-1, 0, -1};
  int lo = 0, hi = c.B;  // first b with cu[b+1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo == c.B || cu[lo] > t) return r;  // behind the last sequence
  const int end = cu[lo + 1];
  if (cu[lo] < 0 || end > rows) return r;  // a sequence that does not fit the rows: recorded by its caller
  const long long pos = static_cast<long long>(c.seq_lens[lo]) - end + t;
  if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) {
    record_status(status, kStatusInvalid, kSitePagedLength);
    return r;
  }
  const int page =
      c.page_table[static_cast<size_t>(lo) * c.max_pages + static_cast<size_t>(pos >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    record_status(status, kStatusInvalid, kSitePagedPage);
    return r;
  }
  r.page = page;
  r.pos = static_cast<int>(pos);
  r.offset = r.pos & ((1 << c.page_shift) - 1);
  return r;
}

// Two e4m3 bytes -> two halves, exactly (e4m3 fits fp16).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Eight e2m1 codes -> four pairs of halves, pair i from byte i (low nibble
// first), exactly.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace fa
