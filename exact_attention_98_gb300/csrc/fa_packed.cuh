// Shared by the kernels of packed sequences: the layout of a plan.
//
// Packed sequences are rows of one tensor, sequence b the rows cu[b] ..
// cu[b+1]-1.  A plan is what the kernels need to know about them, made once from
// cu by one kernel (fa_packed.cu) and used by every call on rows of the same
// batch: a head, each row's position, and three lists of tiles.  A list's entry is
//   {first row of the sequence, its length, the tile's index in it, 0}
//   tiles      128-row tiles, those that see the most keys first
//   blocks     256-row blocks in the same order
//   seq_tiles  128-row tiles, sequence by sequence, those of most tiles first
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

// Work item of the backward: a key tile of a key head, or (split_parts > 1) one
// of as many parts of its query tiles.  The heads (and parts) of an entry of a
// list follow one another.  The list is seq_tiles, so that CTAs that run at the
// same time walk the same query tiles, whose Q, dO and dQ then pass through L2
// once for all of them: 131072 rows of 24 sequences (H = 16, Hkv = 4, d = 128, causal)
// take 5926 us, with the heaviest key tiles of all sequences first 8286.  A causal
// batch of few tiles takes the heaviest first all the same: there the last CTAs' idle
// time weighs more (16384 rows of 11 sequences: 325 us instead of 338, both with a
// sequence's heads in turn).  The limit counts tiles, not items (tiles times key heads),
// and lies between two batches measured, both of 4 key heads: these 132 tiles and those
// of 131072 rows, more than 1000.  Where it lies for 1 or 16 key heads is not known.
constexpr int kFewTiles = 152;
struct PackedItem {
  int start, len;  // rows of the sequence
  int kt;          // key tile
  int kv;          // key head
  bool causal;
};

// Items of a backward call, without their parts: 0 when the plan is not one for its
// rows (recorded).
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
  const PackedHead& h = *static_cast<const PackedHead*>(p.plan);
  // in `tiles` the last tile of a sequence costs most; its first key tile does
  const bool heaviest = h.causal != 0 && h.n_tiles <= kFewTiles;
  const int entry = p.div_kv.div(i);
  const int4 e = (heaviest ? p.tiles : p.seq_tiles)[entry];
  PackedItem it;
  it.start = e.x;
  it.len = e.y;
  it.kv = i - entry * p.BH;
  it.kt = heaviest ? (e.y - 1) / kBlockN - e.z : e.z;
  it.causal = h.causal != 0;
  return it;
}

// The item of block blk, and its part (-1: not split).
__device__ __forceinline__ int packed_block(const BwdParams& p, int blk, int& part) {
  part = -1;
  if (p.split_parts == 1) return blk;
  const int i = p.div_parts.div(blk);
  part = blk - i * p.split_parts;
  return i;
}

// fp32 dK or dV (unscaled) of a part: [part][dK, dV][key heads][rows][d].
__device__ __forceinline__ float* packed_part(const BwdParams& p, int part, bool dv, int kv, int row, int d) {
  return p.tile_part + (((static_cast<size_t>(part) * 2 + (dv ? 1 : 0)) * p.BH + kv) * p.N + row) * d;
}
// 64 columns of such a row; `some`: the part has query tiles, else they are zeros.
__device__ __forceinline__ void packed_part_row(float* to, const uint32_t (&r)[2][32], bool some) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t* x = &r[c >> 2][(c & 3) * 8];
    if (some)
      st_global_v8(to + 8 * c, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
    else
      st_global_v8(to + 8 * c, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u);
  }
}

}  // namespace fa
