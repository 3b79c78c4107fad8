// Shared by the kernels of packed sequences: the layout of a plan.
//
// Packed sequences are rows of one tensor, sequence b the rows cu[b] ..
// cu[b+1]-1.  A plan is what the kernels need to know about them, made once from
// cu by one kernel (fa_packed.cu) and used by every call on rows of the same
// batch: a head, each row's position, and three lists of tiles.  A list's entry is
//   {first row of the sequence, its length, the tile's index in it, w}
//   tiles      128-row tiles, those that see the most keys first
//   blocks     256-row blocks in the same order
//   seq_tiles  128-row tiles, sequence by sequence, those of most tiles first;
//              w is the index in this list of the sequence's first
#pragma once

#include "fa_device.cuh"
#include "fa_kernels.h"

namespace fa {

constexpr int kPackedMagic = 0x3198fa50;
constexpr size_t kPackedHeadBytes = 256;

struct PackedHead {
  int magic;
  int rows;       // of the tensors
  int sequences;
  int causal;
  int n_tiles;    // entries of tiles and of seq_tiles
  int n_blocks;   // entries of blocks
  int begin, end;  // rows of the first sequence's start and of the last one's end
};

// Entries of a list of tiles of `size` rows at most: every sequence with rows
// ends in one tile that is not full.
__host__ __device__ constexpr long long packed_tiles(long long rows, long long sequences, int size) {
  return rows / size + (rows < sequences ? rows : sequences);
}

// Byte offsets within a plan, each a multiple of 256.
struct PackedLayout {
  size_t positions, tiles, blocks, seq_tiles, bytes;
};
__host__ __device__ constexpr size_t packed_round(size_t x) { return (x + 255) / 256 * 256; }
__host__ __device__ constexpr PackedLayout packed_layout(long long rows, long long sequences) {
  PackedLayout l{};
  const size_t tiles = packed_round(static_cast<size_t>(packed_tiles(rows, sequences, kBlockM)) * sizeof(int4));
  const size_t blocks = packed_round(static_cast<size_t>(packed_tiles(rows, sequences, 2 * kBlockM)) * sizeof(int4));
  l.positions = kPackedHeadBytes;
  l.tiles = l.positions + packed_round(static_cast<size_t>(rows) * sizeof(int));
  l.blocks = l.tiles + tiles;
  l.seq_tiles = l.blocks + blocks;
  l.bytes = l.seq_tiles + tiles;
  return l;
}

// Site codes recorded with FA_ERR_INVALID_ARG.
constexpr unsigned int kPackedInvalid = 1u;
enum : unsigned int {
  kSitePackedOffsets = 0x701,   // cu does not run forwards within the rows
  kSitePackedPlan = 0x702,      // not a plan, or one for other rows or sequences
  kSitePackedPosition = 0x703,  // a position past the rotation's table
};

// Whether the plan is one for this call's rows.
__device__ __forceinline__ bool packed_fits(const PackedHead& h, int rows, int sequences) {
  return h.magic == kPackedMagic && h.rows == rows && h.sequences == sequences;
}

// Work item of the backward: a key tile of a key head.  Item i belongs to the
// sequence of entry i / Hkv of seq_tiles; within a sequence the heads come one
// after another, the key tiles of each in order (causal: those of most work first), so
// that CTAs that run at the same time add to the same rows of dQ.
struct PackedItem {
  int start, len;  // rows of the sequence
  int kt;          // key tile
  int kv;          // key head
  bool causal;
};

// Items of a backward call: 0 when the plan is not one for its rows (recorded).
__device__ __forceinline__ int packed_items(const BwdParams& p) {
  const PackedHead& h = *static_cast<const PackedHead*>(p.plan);
  if (!packed_fits(h, p.N, p.sequences)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_status(p.status, kPackedInvalid, kSitePackedPlan);
    return 0;
  }
  return h.n_tiles * p.BH;
}

// Item i (< packed_items) of a backward call.
__device__ __forceinline__ PackedItem packed_item_at(const BwdParams& p, int i) {
  const uint8_t* plan = static_cast<const uint8_t*>(p.plan);
  const int4 e = reinterpret_cast<const int4*>(plan + packed_layout(p.N, p.sequences).seq_tiles)[p.div_kv.div(i)];
  PackedItem it;
  it.start = e.x;
  it.len = e.y;
  const int tiles = (e.y + kBlockN - 1) / kBlockN, at = i - e.w * p.BH;
  it.kv = at / tiles;
  it.kt = at - it.kv * tiles;
  it.causal = reinterpret_cast<const PackedHead*>(plan)->causal != 0;
  return it;
}
__device__ __forceinline__ bool packed_item(const BwdParams& p, int i, PackedItem& it) {
  if (i >= packed_items(p)) return false;
  it = packed_item_at(p, i);
  return true;
}

}  // namespace fa
