// Attention of each sequence's last tokens over its paged key/value cache.
//
// The token at position p of a sequence sees the cached positions j <= p with
// p - j < window, and the first `sinks` positions: S_j = scale q.k_j over
// these, O = softmax(S) V, LSE = ln sum exp S_j.
//
// Bound by HBM: each visible cached row is read once per key head and serves
// every query head of the group.  The products are narrow (8 or 16 pairs of a
// row and a head of the group at a time), far below the tensor cores' rate,
// and their operands come from registers, where a 4-bit row is turned into
// halves anyway, so mma.sync carries them, transposed: cached positions (Q K^T)
// and d (P V) are the products' 16 rows, and the pairs their 8 columns, so that
// no product is spent on empty rows.
//
// Work: a segment is (sequence, key head, block of 8 kTiles rows) and a list of
// units of 64 (bf16: 16) positions: those of the first tokens, then those of
// the window.  All units of all segments are laid out in one line, which
// the grid's warps cut into equal pieces, whatever the lengths of the
// sequences (read on the device, so that a captured graph serves any
// lengths).  A warp that holds the whole of a segment writes its rows; the
// parts of a segment that several warps share go to the workspace (at most
// two parts per warp), and a second kernel joins them by their maxima and
// sums.  Warps share nothing else: each copies its units' rows into a ring of
// its own in shared memory, one or two units ahead of its products, bf16 by tiled TMA
// with the 128-byte swizzle that ldmatrix reads without conflicts, 4-bit codes
// and scales as plain bulk copies.
//
// 4 bits: codes become halves exactly (e2m1 x e4m3 has six bits), so the only
// roundings are those of P to fp16 and of the result.  Q is scaled to fp16
// by a power of two per row.  The products are free to permute d: lane
// (g, c) of a warp reads of keys g and g + 8 the codes [c D/4, (c+1) D/4) in one
// load each, and of the keys 2c, 2c+1, 2c+8, 2c+9 (V) the codes [g D/8, (g+1) D/8).
//
// Measured (d = 128): 4 bits, 32 sequences of up to 32768 positions, 8 key and 32
// query heads, one token each: 142 us, 5.4 TB/s of 6.7; the FMA and ALU work of
// the codes issues 64% of the slots and bounds it beside HBM (units of 32
// positions: 175 us).  48 sequences, 3 new tokens, a window of 4096: 46 us, 2.5
// TB/s, of which about 16 are the launches, the tables, the first copies and the
// join; 12 pairs are two tiles, 253 registers, 8 warps to an SM.  bf16, 32 such
// sequences, L2 flushed: 389 us, 6.2 TB/s (d = 64: 209, 5.8); one
// sequence of 4097 positions: 15 us on the GPU, the same fixed cost.
// kTiles: one where no block has more than 8 pairs (two there: 194 instead of
// 142 us), else two (one, which reads the rows twice: 60 instead of 46).
#include <limits.h>

#include "fa_paged.cuh"

namespace fa {
namespace {

enum : unsigned int {
  kSitePagedFull = 0x511,
};

// A running reference is set kBelow (log2 units) below the maximum at hand, and
// the sums and accumulators are rescaled once a score is kSlack above that
// maximum.  bf16 keeps the dominant weight near 1 (its rounding error reaches O)
// and has exponents enough for the small ones.  fp16's spacing is 8 times finer
// but ends at 2^-24: with the largest weight at 2^7 to 2^15 a weight is held
// down to 2^-32 of it, so that a long tail under one dominating position counts
// in O as it does in the sum (with kBelow = 0, 2^17 positions at 2^-25 were lost).
template <bool FP4>
__device__ constexpr float kSlack = FP4 ? 8.0f : 2.0f;
template <bool FP4>
__device__ constexpr float kBelow = FP4 ? 7.0f : 0.0f;

template <int D, bool FP4, int TILES>
struct PagedCfg {
  static constexpr int kRows = 8 * TILES;            // rows of a block
  static constexpr int kUnitShift = FP4 ? 6 : 4;
  static constexpr int kUnit = 1 << kUnitShift;      // positions of a unit
  static constexpr int kLeast = 64 / kUnit;          // units of a warp's piece at least
  static constexpr int kWarps = FP4 ? (TILES == 2 ? 8 : 12) : 8;
  static constexpr int kCtas = 1;  // per SM
  static constexpr int kWorkers = kWarps * kCtas;    // warps per SM
  static constexpr int kStages = FP4 ? (TILES == 2 ? 3 : 2) : 3;
  static constexpr int kRowBytes = FP4 ? D / 2 + D / 16 : 2 * D;
  static constexpr int kHalf = kUnit * kRowBytes;    // K rows of a unit
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kBarOff = kWarps * kStages * kStageBytes;
  static constexpr int kStartOff = kBarOff + kWarps * kStages * 8;  // [warps] {sequence, offset}
  static constexpr int kScanOff = kStartOff + kWarps * 16;
  static constexpr int kAbortOff = kScanOff + kWarps * 8;
  static constexpr int kSmemBytes = kAbortOff + 16 + 1024;
  static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
};

// What a sequence asks for.
struct Seq {
  int row0, n;      // its rows of q
  int len;          // cached positions
  int first;        // units of the first tokens
  int skip;         // the window's first unit, less `first`
  int units;        // units of a segment: its loads, or 1 without any
  int loads;        // units that hold positions
  int blocks;       // blocks of rows
  int lo;           // the first position that the window of its rows reaches
};

template <class C>
__device__ __forceinline__ Seq paged_seq(const FwdPagedParams& p, int b, bool report) {
  Seq s;
  const int r0 = p.cu[b], r1 = p.cu[b + 1];
  const bool bad = r0 < 0 || r1 < r0 || r1 > p.rows;
  s.row0 = r0;
  s.n = bad ? 0 : min(r1 - r0, p.max_new);  // rows past max_new: not computed
  const int extra = bad ? 0 : r1 - r0 - s.n;
  if (report && (bad || extra > 0)) record_status(p.status, kStatusInvalid, kSitePagedRows);
  const long long most = static_cast<long long>(p.c.max_pages) << p.c.page_shift;
  s.len = p.c.seq_lens[b];
  if (s.len < 0 || s.len > most) {  // no telling where its rows are: they see nothing
    if (report) record_status(p.status, kStatusInvalid, kSitePagedLength);
    s.len = 0;
  }
  s.len = max(0, s.len - extra);
  const int end = (s.len + C::kUnit - 1) / C::kUnit;
  s.lo = p.window == INT_MAX ? 0 : max(0, max(0, s.len - s.n) - p.window + 1);
  const int win = s.lo / C::kUnit;
  s.first = min((min(p.sinks, s.len) + C::kUnit - 1) / C::kUnit, win);
  s.skip = win - s.first;
  s.loads = s.n > 0 ? end - s.skip : 0;
  s.units = max(1, s.loads);
  s.blocks = (s.n * p.group + C::kRows - 1) / C::kRows;
  return s;
}

__device__ __forceinline__ long long seq_units(const FwdPagedParams& p, const Seq& s) {
  return static_cast<long long>(s.units) * s.blocks * p.c.Hkv;
}

// A warp's place in the line of units.
struct Walk {
  int left;  // units left to this warp
  int b;     // sequence
  int seg;   // key head * blocks + block of rows
  int unit;  // within the segment
  Seq s;
};

// Moves to the next segment after `done` units of this one.
template <class C>
__device__ __forceinline__ void walk_next(const FwdPagedParams& p, Walk& w, int done) {
  w.left -= done;
  w.unit = 0;
  if (++w.seg < w.s.blocks * p.c.Hkv) return;
  w.seg = 0;
  while (w.left > 0 && w.b + 1 < p.c.B) {
    w.s = paged_seq<C>(p, ++w.b, false);
    if (w.s.blocks > 0) return;
  }
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// This warp's copies: the units of its piece in order, each into the next stage.
template <int D, bool FP4, int TILES>
struct Loader {
  using C = PagedCfg<D, FP4, TILES>;
  Walk w;
  // Page numbers come 32 at a time, one per lane: a batch of 32 units, or fewer
  // where a unit spans several pages.  A lane keeps where its page's part of the
  // unit starts: 4 bits, the address of its K codes (null: nothing to copy);
  // bf16, block * 2 (-1: nothing).
  unsigned long long at;
  int batch;   // units of the batch left, 0: to be loaded
  int stage;   // the next copy's
  // Parts of a stage that were not copied, 4 bits a stage: bit i the unit's i-th
  // page (0 where a page holds the whole unit).  The stage keeps what it held there.
  unsigned int holes;

  __device__ __forceinline__ void next(const FwdPagedParams& p, uint32_t ring, uint32_t bars, int lane) {
    if (w.left <= 0) return;
    while (w.unit >= w.s.loads) {  // a segment's end, or one without positions
      walk_next<C>(p, w, w.s.loads == 0 ? 1 : 0);
      batch = 0;
      if (w.left <= 0) return;
    }
    const int shift = min(p.c.page_shift, C::kUnitShift);  // positions of a page within a unit
    const int subs_shift = C::kUnitShift - shift;
    const int first_key = (w.unit < w.s.first ? w.unit : w.unit + w.s.skip) * C::kUnit;
    const int page_mask = (1 << p.c.page_shift) - 1;
    if (batch == 0) {
      batch = 32 >> subs_shift;
      const int u = w.unit + (lane >> subs_shift);
      const int key = (u < w.s.first ? u : u + w.s.skip) * C::kUnit + ((lane & ((1 << subs_shift) - 1)) << shift);
      at = FP4 ? 0ull : ~0ull;
      // (a page of a unit that no row of the sequence sees may have been given back)
      const bool seen = key < p.sinks || key + (1 << shift) > w.s.lo;
      if (u < w.s.loads && u < w.unit + w.left && key < w.s.len && seen) {
        const int page = p.c.page_table[static_cast<size_t>(w.b) * p.c.max_pages + (key >> p.c.page_shift)];
        if (page < 0 || page >= p.c.num_pages) {
          record_status(p.status, kStatusInvalid, kSitePagedPage);
        } else {
          const size_t block2 = (static_cast<size_t>(page) * p.c.Hkv + w.seg / w.s.blocks) * 2;
          at = block2;
          if constexpr (FP4)
            at = reinterpret_cast<unsigned long long>(p.c.pages) +
                 block2 * paged_half_bytes(true, 1 << p.c.page_shift, D) +
                 static_cast<unsigned int>((key & page_mask) * (D / 2));
        }
      }
    }
    const uint32_t dst = ring + stage * C::kStageBytes;
    const uint32_t bar = bars + 8 * stage;
    // 4 bits: a lane per page of the unit, whose block is one copy; a page
    // longer than the unit: lanes 0-3, its part of K's and V's codes and scales.
    // bf16: lanes 0-3, K and V, 64 columns each.
    const bool parts = !FP4 || p.c.page_shift > C::kUnitShift;
    const int sub = parts ? 0 : lane & ((1 << subs_shift) - 1);
    const unsigned long long from =
        __shfl_sync(0xffffffffu, at, (((32 >> subs_shift) - batch) << subs_shift) + sub);
    const bool mine = lane < (parts ? 4 : 1 << subs_shift) && from != (FP4 ? 0ull : ~0ull);
    const unsigned int live = __ballot_sync(0xffffffffu, mine);
    const unsigned int hole = parts ? (live == 0u ? 1u : 0u) : ~live & ((1u << (1 << subs_shift)) - 1u);
    holes = (holes & ~(15u << (4 * stage))) | (hole << (4 * stage));
    if (lane == 0)
      mbar_arrive_expect_tx(bar, __popc(live) * (parts ? C::kStageBytes / 4 : C::kStageBytes >> subs_shift));
    __syncwarp();
    if (mine) {
      const int kv = (lane >> 1) & 1, part = lane & 1;
      if constexpr (FP4) {
        if (!parts) {
          const uint32_t bytes = C::kStageBytes >> subs_shift;
          bulk_load(dst + sub * bytes, reinterpret_cast<const uint8_t*>(from), bytes, bar);
        } else {
          const uint32_t half = static_cast<uint32_t>(paged_half_bytes(true, 1 << p.c.page_shift, D));
          // the scales of a row stand behind the page's codes
          const uint32_t in_page = first_key & page_mask;
          const uint32_t src = kv * half + (part ? ((D / 2) << p.c.page_shift) - in_page * (D / 2 - D / 16) : 0u);
          bulk_load(dst + kv * C::kHalf + (part ? C::kUnit * (D / 2) : 0),
                    reinterpret_cast<const uint8_t*>(from) + src, C::kUnit * (part ? D / 16 : D / 2), bar);
        }
      } else if (part < D / 64) {
        tma_load_3d(dst + kv * C::kHalf + part * (C::kUnit * 128), &p.tm, bar, part * 64, first_key & page_mask,
                    static_cast<int>(from) + kv);
      }
    }
    stage = stage == C::kStages - 1 ? 0 : stage + 1;
    --batch;
    ++w.unit;
    --w.left;
  }
};

template <int D, bool FP4, int TILES>
__global__ void __launch_bounds__(32 * PagedCfg<D, FP4, TILES>::kWarps, PagedCfg<D, FP4, TILES>::kCtas)
    fa_fwd_paged_kernel(const __grid_constant__ FwdPagedParams p) {
  using C = PagedCfg<D, FP4, TILES>;
  constexpr int kSteps = D / 16;  // k16 steps of Q K^T, and m16 tiles of P V
  constexpr int kGroups = C::kUnit / 16;  // k16 steps of P V in a unit
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);
  const WaitCtl ctl{abort_flag, p.status};
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::kWarps * C::kStages; ++s) mbar_init(sbase + C::kBarOff + 8 * s, 1);
    fence_mbar_init();
  }
  grid_dependency_wait();
  __syncthreads();

  // ---- this warp's piece of the line of units
  long long* scan = reinterpret_cast<long long*>(smem + C::kScanOff);
  long long* start = reinterpret_cast<long long*>(smem + C::kStartOff);
  auto block_scan = [&](long long v, long long& total) {  // inclusive, over the CTA's threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    total = 0;
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) v += scan[w];
      total += scan[w];
    }
    return v;
  };
  long long total = 0, mine = 0, end = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32 * C::kWarps) {
    const int b = b0 + threadIdx.x;
    long long t;
    mine = b < p.c.B ? seq_units(p, paged_seq<C>(p, b, blockIdx.x == 0)) : 0;
    end = total + block_scan(mine, t);
    total += t;
  }
  // worker i: warp i / grid of CTA i % grid, so that few units spread over the SMs
  const int grid = static_cast<int>(gridDim.x);
  const long long workers =
      max(1LL, min(static_cast<long long>(grid) * C::kWarps, (total + C::kLeast - 1) / C::kLeast));
  const long long quot = total <= 0x7fffffffLL
                             ? static_cast<long long>(static_cast<unsigned int>(total) / static_cast<unsigned int>(workers))
                             : total / workers;
  const long long rem = total - quot * workers;
  auto piece = [&](long long i) { return quot * i + min(i, rem); };
  const long long me = static_cast<long long>(warp) * grid + blockIdx.x;
  const bool once = p.c.B <= 32 * C::kWarps;  // the scan above still holds every sequence
  long long before = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32 * C::kWarps) {
    const int b = b0 + threadIdx.x;
    if (!once) {
      long long t;
      mine = b < p.c.B ? seq_units(p, paged_seq<C>(p, b, false)) : 0;
      end = before + block_scan(mine, t);
      before += t;
    }
    for (int w = 0; w < C::kWarps; ++w) {
      const long long i = static_cast<long long>(w) * grid + blockIdx.x;
      const long long u0 = piece(i);
      if (i < workers && u0 < end && u0 >= end - mine) {
        start[2 * w] = b;
        start[2 * w + 1] = u0 - (end - mine);
      }
    }
  }
  __syncthreads();
  if (lane == 0) p.info[me] = make_int4(0, 0, 0, 0);
  if (me >= workers || total == 0) return;
  Walk w;
  w.left = static_cast<int>(piece(me + 1) - piece(me));
  w.b = static_cast<int>(start[2 * warp]);
  w.s = paged_seq<C>(p, w.b, false);
  // (a sequence's units: sized by its row of the page table, times its segments)
  const long long at = start[2 * warp + 1];
  w.seg = at <= 0x7fffffffLL ? static_cast<int>(static_cast<unsigned int>(at) / static_cast<unsigned int>(w.s.units))
                             : static_cast<int>(at / w.s.units);
  w.unit = static_cast<int>(at - static_cast<long long>(w.seg) * w.s.units);

  const uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_s = sbase + warp * C::kStages * C::kStageBytes;
  const uint32_t bars = sbase + C::kBarOff + warp * C::kStages * 8;
  Loader<D, FP4, TILES> load;
  load.w = w;
  load.batch = 0;
  load.at = 0;
  load.stage = 0;
  load.holes = 0u;
  for (int i = 0; i < C::kStages; ++i) load.next(p, ring_s, bars, lane);

  const int g = lane >> 2, c = lane & 3;
  // 4 bits: a stage holds blocks of sub_keys positions as the cache does (K codes,
  // K scales, V codes, V scales)
  const int sub_shift = min(p.c.page_shift, C::kUnitShift);
  const int sub_half = paged_half_bytes(FP4, 1 << sub_shift, D);
  int stage = 0;
  uint32_t parity = 0;
  bool ok = true;
  while (w.left > 0) {
    const int kvh = w.seg / w.s.blocks;
    const int block = w.seg - kvh * w.s.blocks;
    const int u1 = min(w.s.units, w.unit + w.left);
    const int n_load = min(u1, w.s.loads);
    const int n_pairs = w.s.n * p.group;
    const int pair0 = block * C::kRows;
    const int pos0 = w.s.len - w.s.n;  // position of the first new row
    // the block's rows' positions, least and most
    const int p_lo = max(-1, pos0 + pair0 / p.group);
    const int p_hi = max(-1, pos0 + (min(n_pairs, pair0 + C::kRows) - 1) / p.group);

    // Q as the products' B operand: lane (g, c) holds of pair g the elements
    // (4 bits) c D/4 + 4 s + {0, 1} and + {2, 3}, (bf16) 16 s + 2c + {0, 1} and + 8
    uint32_t qb[TILES][kSteps][2];
    float mul[TILES][2];  // of pairs 2c, 2c + 1, as the scores have them
    int pos[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int pair = pair0 + t * 8 + g;
      const int tok = pair / p.group;
      const bool in = pair < n_pairs;
      const __nv_bfloat16* src = p.q + (w.s.row0 + static_cast<long long>(in ? tok : 0)) * p.q_row +
                                 (kvh * p.group + (pair - tok * p.group)) * p.q_head;
      float f = p.scale;
      if constexpr (FP4) {
        uint4 raw[D / 32];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (in) raw[i] = *reinterpret_cast<const uint4*>(src + c * (D / 4) + 8 * i);
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // a power of two brings the row's largest magnitude into [1, 2):
        // down is 2^-e, f takes its inverse (both kept in the normal range)
        const int e = min(253, max(1, static_cast<int>((__float_as_uint(amax) >> 23) & 255u)));
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        f *= __uint_as_float(static_cast<uint32_t>(e) << 23);
        if (p.c.k_scale) f *= p.c.k_scale[kvh];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            qb[t][2 * i + (k >> 1)][k & 1] =
                pack_f16x2(__uint_as_float(x[k] << 16) * down, __uint_as_float(x[k] & 0xFFFF0000u) * down);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qb[t][k][u] = in ? *reinterpret_cast<const uint32_t*>(src + k * 16 + u * 8 + 2 * c) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mul[t][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + e));
        const int pr = pair0 + t * 8 + 2 * c + e;
        pos[t][e] = pr < n_pairs ? max(-1, pos0 + pr / p.group) : -1;
      }
    }

    float acc[TILES][kSteps][4];
    float ref[TILES][2], lim[TILES][2], l[TILES][2];  // reference (log2 units), how far above it is too far, sums
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][j][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[t][e] = 0.0f;
        lim[t][e] = -INFINITY;  // nothing seen yet: any score moves the reference
        l[t][e] = 0.0f;
      }
    }

    for (int u = w.unit; u < n_load; ++u) {
      if (ok && !mbar_wait_warp(bars + 8 * stage, parity, ctl, kSitePagedFull)) {
        // given up: no more copies; those in flight (this stage's and the ones
        // after it) land before shared memory is released
        ok = false;
        for (int i = 0; i < C::kStages; ++i)
          mbar_wait_drain(bars + 8 * ((stage + i) % C::kStages), parity ^ (stage + i >= C::kStages ? 1u : 0u));
      }
      const int unit_key = (u < w.s.first ? u : u + w.s.skip) * C::kUnit;
      const uint8_t* st = ring + stage * C::kStageBytes;
      const uint32_t st_s = ring_s + stage * C::kStageBytes;
      const unsigned int hole = (load.holes >> (4 * stage)) & 15u;
      // every position there, and visible to every row?
      const bool edge = hole != 0u || unit_key + C::kUnit - 1 > p_lo ||
                        (unit_key < p_hi - p.window + 1 && unit_key + C::kUnit > p.sinks);
      // S^T = K Q^T: key unit_key + 16 grp + g (0, 1) or + 8 (2, 3) of pairs 2c, 2c + 1
      float s[kGroups][TILES][4];
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[grp][t][e] = 0.0f;
        if constexpr (FP4) {
          const uint8_t* k_rows = st + ((grp * 16) >> sub_shift) * 2 * sub_half;
          const int in_block = (grp * 16) & ((1 << sub_shift) - 1);
          uint32_t codes[2][D / 32];
          uint32_t sc[2][D / 64];  // the scales of this lane's blocks of 16, twice each
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            const int row = in_block + k8 * 8 + g;
            const uint8_t* kc = k_rows + row * (D / 2) + c * (D / 8);
            const uint8_t* ks = k_rows + ((D / 2) << sub_shift) + row * (D / 16) + c * (D / 64);
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(kc);
              codes[k8][0] = x.x; codes[k8][1] = x.y; codes[k8][2] = x.z; codes[k8][3] = x.w;
              const uint32_t two = *reinterpret_cast<const unsigned short*>(ks);
              const uint32_t h = e4m3x2_to_f16x2(two);
              sc[k8][0] = __byte_perm(h, 0u, 0x1010);
              sc[k8][1] = __byte_perm(h, 0u, 0x3232);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kc);
              codes[k8][0] = x.x; codes[k8][1] = x.y;
              sc[k8][0] = e4m3x2_to_f16x2(*ks * 0x101u);
            }
          }
#pragma unroll
          for (int wd = 0; wd < D / 32; ++wd) {
            uint32_t x[4], y[4];
            e2m1x8_to_f16x2(codes[0][wd], x);
            e2m1x8_to_f16x2(codes[1][wd], y);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {hmul2(x[2 * k], sc[0][wd >> 1]), hmul2(y[2 * k], sc[1][wd >> 1]),
                                     hmul2(x[2 * k + 1], sc[0][wd >> 1]), hmul2(y[2 * k + 1], sc[1][wd >> 1])};
#pragma unroll
              for (int t = 0; t < TILES; ++t) mma16816<true>(s[grp][t], a, qb[t][2 * wd + k]);
            }
          }
        } else {
          // lanes 0-15: keys 0-15, the first 8 of 16 elements; 16-31: the other 8
          const int row = grp * 16 + (lane & 15);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t a[4];
            const int chunk = (k & 3) * 2 + (lane >> 4);
            ldmatrix_x4(st_s + (k >> 2) * (C::kUnit * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), a);
#pragma unroll
            for (int t = 0; t < TILES; ++t) mma16816<false>(s[grp][t], a, qb[t][k]);
          }
        }
      }

      // scores relative to the references
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp)
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[grp][t][e] = fmaf(s[grp][t][e], mul[t][e & 1], -ref[t][e & 1]);
      // Masked scores are -inf.  A position that no row sees has weight 0, but
      // its row of V may hold anything (the rest of a page, infinities): it is
      // zeroed.  Bit 4 grp + k of keep: position 16 grp + 2c + {0, 1, 8, 9}[k].
      unsigned int keep = 0xFFFFu;
      if (edge) {
        keep = 0u;
#pragma unroll 1
        for (int grp = 0; grp < kGroups; ++grp) {
          const int key0 = unit_key + grp * 16;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = key0 + (k >> 1) * 8 + 2 * c + (k & 1);
            if (j <= p_hi && (j < p.sinks || j > p_lo - p.window)) keep |= 1u << (4 * grp + k);
          }
        }
#pragma unroll
        for (int grp = 0; grp < kGroups; ++grp)
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = unit_key + grp * 16 + g + (e >> 1) * 8;
              const int q = pos[t][e & 1];
              if (j > q || (j <= q - p.window && j >= p.sinks)) s[grp][t][e] = -INFINITY;
            }
        // pages outside the cache: no row sees their positions
#pragma unroll
        for (int grp = 0; grp < kGroups; ++grp)
          if ((hole >> ((grp * 16) >> sub_shift)) & 1u) {
            keep &= ~(15u << (4 * grp));
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[grp][t][e] = -INFINITY;
          }
      }
      bool over = false;
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[0][t][e], s[0][t][e + 2]);
#pragma unroll
          for (int grp = 1; grp < kGroups; ++grp) mx = fmax3(mx, s[grp][t][e], s[grp][t][e + 2]);
          over = over || mx > lim[t][e];
        }
      if (__any_sync(0xffffffffu, over)) {
        // some reference is too far below: all that are behind move up
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[0][t][e], s[0][t][e + 2]);
#pragma unroll
            for (int grp = 1; grp < kGroups; ++grp) mx = fmax3(mx, s[grp][t][e], s[grp][t][e + 2]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (mx > lim[t][e]) {
              const float up = mx - kBelow<FP4>;
              const float a = lim[t][e] == -INFINITY ? 0.0f : ex2_mufu(-up);
              ref[t][e] += up;
              lim[t][e] = kSlack<FP4> + kBelow<FP4>;
#pragma unroll
              for (int grp = 0; grp < kGroups; ++grp) {
                s[grp][t][e] -= up;
                s[grp][t][e + 2] -= up;
              }
              l[t][e] *= a;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                acc[t][j][e] *= a;
                acc[t][j][e + 2] *= a;
              }
            }
          }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) {
        uint32_t pb[TILES][2];  // P as the B operand: keys 2c, 2c + 1 (and + 8) of pair g
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            const float x = ex2_mufu(s[grp][t][2 * k8]), y = ex2_mufu(s[grp][t][2 * k8 + 1]);
            l[t][0] += x;
            l[t][1] += y;
            pb[t][k8] = transpose8x8(FP4 ? pack_f16x2(x, y) : pack_bf16x2(x, y));
          }
        if constexpr (FP4) {
          // rows g, g + 8 of m-tile j are d = g D/8 + 2j, + 1
          const uint8_t* v_rows = st + (((grp * 16) >> sub_shift) * 2 + 1) * sub_half;
          const int in_block = (grp * 16) & ((1 << sub_shift) - 1);
          const uint8_t* vc = v_rows + (in_block + 2 * c) * (D / 2) + g * (D / 16);
          const uint8_t* vs = v_rows + ((D / 2) << sub_shift) + (in_block + 2 * c) * (D / 16) + (g * D) / 128;
          uint32_t sc[2];  // scales of the keys' pairs
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            uint32_t two = vs[k8 * 8 * (D / 16)] | (static_cast<uint32_t>(vs[(k8 * 8 + 1) * (D / 16)]) << 8);
            if (edge) {
              const unsigned int bits = keep >> (4 * grp + 2 * k8);
              two &= ((bits & 1u) ? 0xFFu : 0u) | ((bits & 2u) ? 0xFF00u : 0u);
            }
            sc[k8] = e4m3x2_to_f16x2(two);
          }
          uint32_t codes[2][2][D / 64];  // [+0, +8][key][word]
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint8_t* at = vc + (k8 * 8 + k) * (D / 2);
              if constexpr (D == 128) {
                const uint2 x = *reinterpret_cast<const uint2*>(at);
                codes[k8][k][0] = x.x;
                codes[k8][k][1] = x.y;
              } else {
                codes[k8][k][0] = *reinterpret_cast<const uint32_t*>(at);
              }
            }
#pragma unroll
          for (int wd = 0; wd < D / 64; ++wd) {
            uint32_t even[2][4], odd[2][4];
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8) {
              const uint32_t a = codes[k8][0][wd], b = codes[k8][1][wd];
              // byte i: element 2i (or 2i + 1), of the even key low, of the odd key high
              e2m1x8_to_f16x2((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), even[k8]);
              e2m1x8_to_f16x2(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), odd[k8]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a[4] = {hmul2(even[0][k], sc[0]), hmul2(odd[0][k], sc[0]), hmul2(even[1][k], sc[1]),
                                     hmul2(odd[1][k], sc[1])};
#pragma unroll
              for (int t = 0; t < TILES; ++t) mma16816<true>(acc[t][wd * 4 + k], a, pb[t]);
            }
          }
        } else {
          // rows g, g + 8 of m-tile j are d = 16 j + g, + 8: lanes 0-7 keys 0-7 of
          // columns 16j.., 8-15 the next 8 columns, 16-31 keys 8-15
          const int row = grp * 16 + (lane & 7) + ((lane >> 4) << 3);
          const unsigned int bits = keep >> (4 * grp);
          const uint32_t k01 = ((bits & 1u) ? 0xFFFFu : 0u) | ((bits & 2u) ? 0xFFFF0000u : 0u);
          const uint32_t k89 = ((bits & 4u) ? 0xFFFFu : 0u) | ((bits & 8u) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            uint32_t a[4];
            const int chunk = (j & 3) * 2 + ((lane >> 3) & 1);
            ldmatrix_x4_t(st_s + C::kHalf + (j >> 2) * (C::kUnit * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), a);
            if (edge) {
              a[0] &= k01; a[1] &= k01; a[2] &= k89; a[3] &= k89;
            }
#pragma unroll
            for (int t = 0; t < TILES; ++t) mma16816<false>(acc[t][j], a, pb[t]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (ok) load.next(p, ring_s, bars, lane);
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }

    // ---- the segment's rows, or this warp's part of them
    const bool whole = w.unit == 0 && u1 == w.s.units;
    const size_t slot = 2 * static_cast<size_t>(me) + (w.unit == 0 ? 1 : 0);
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[t][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float top = lim[t][e] == -INFINITY ? -INFINITY : ref[t][e];
        const int r = t * 8 + 2 * c + e;
        if (!whole) {
          float* out = p.part_o + (slot * C::kRows + r) * D;
          if constexpr (FP4) {
#pragma unroll
            for (int j = 0; j < kSteps; j += 2)
              *reinterpret_cast<float4*>(out + g * (D / 8) + 2 * j) =
                  make_float4(acc[t][j][e], acc[t][j][e + 2], acc[t][j + 1][e], acc[t][j + 1][e + 2]);
          } else {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              out[16 * j + g] = acc[t][j][e];
              out[16 * j + 8 + g] = acc[t][j][e + 2];
            }
          }
          if (g == 0) {
            p.part_ml[slot * 2 * C::kRows + r] = top;
            p.part_ml[slot * 2 * C::kRows + C::kRows + r] = sum;
          }
          continue;
        }
        const int pair = pair0 + r;
        if (pair >= n_pairs) continue;
        const int tok = pair / p.group;
        const size_t at = (static_cast<size_t>(w.s.row0) + tok) * p.H + kvh * p.group + (pair - tok * p.group);
        float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (FP4 && p.c.v_scale) inv *= p.c.v_scale[kvh];
        __nv_bfloat16* out = p.o + at * D;
        if constexpr (FP4) {
          uint32_t x[kSteps];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) x[j] = pack_bf16x2(acc[t][j][e] * inv, acc[t][j][e + 2] * inv);
#pragma unroll
          for (int j = 0; j < kSteps; j += 4)
            *reinterpret_cast<uint4*>(out + g * (D / 8) + 2 * j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            out[16 * j + g] = __float2bfloat16_rn(acc[t][j][e] * inv);
            out[16 * j + 8 + g] = __float2bfloat16_rn(acc[t][j][e + 2] * inv);
          }
        }
        if (g == 0) p.lse[at] = sum == 0.0f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
      }
    if (lane == 0 && w.unit == 0 && !whole) {
      // the segment goes on in the workers after this one: how many
      const int rest = w.s.units - u1;
      int parts = 1;
      for (long long i = me + 1, got = 0; got < rest; ++i, ++parts) got += piece(i + 1) - piece(i);
      p.info[me] = make_int4(parts, w.b, w.seg, 0);
    }
    walk_next<C>(p, w, u1 - w.unit);
  }
}

// Joins the parts of the segments that start in the workers of this block (8 of
// them, blockIdx.x) and go on in the workers after them: the first part is that
// worker's second slot, the others the following workers' first ones.
// blockIdx.y: 32 columns.  A thread takes 4 columns of a row and every
// kGroups-th part.
constexpr int kJoinThreads = 256;
constexpr int kJoinWorkers = 8;

template <int D, bool FP4, int TILES>
__global__ void __launch_bounds__(kJoinThreads) fa_fwd_paged_join_kernel(const __grid_constant__ FwdPagedParams p,
                                                                         int workers) {
  using C = PagedCfg<D, FP4, TILES>;
  constexpr int kGroups = kJoinThreads / (C::kRows * 8);
  __shared__ float4 sx[kGroups][C::kRows * 8];
  __shared__ float2 sml[kGroups][C::kRows * 8];
  const int at = threadIdx.x % (C::kRows * 8), grp = threadIdx.x / (C::kRows * 8);
  const int row = at / 8, d0 = blockIdx.y * 32 + (at % 8) * 4;
  grid_dependency_wait();
  for (int i = 0; i < kJoinWorkers; ++i) {
    const int me = blockIdx.x * kJoinWorkers + i;
    if (me >= workers) return;
    const int4 info = p.info[me];
    if (info.x == 0) continue;
    float m = -INFINITY, l = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;
    for (int k0 = grp; k0 < info.x; k0 += kBatch * kGroups) {
      float mk[kBatch], lk[kBatch];
      float4 y[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = k0 + b * kGroups;
        mk[b] = -INFINITY;
        lk[b] = 0.0f;
        y[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < info.x) {
          const size_t slot = 2 * (static_cast<size_t>(me) + k) + (k == 0 ? 1 : 0);
          mk[b] = p.part_ml[slot * 2 * C::kRows + row];
          lk[b] = p.part_ml[slot * 2 * C::kRows + C::kRows + row];
          y[b] = *reinterpret_cast<const float4*>(p.part_o + (slot * C::kRows + row) * D + d0);
        }
      }
      float top = m;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) top = fmaxf(top, mk[b]);
      // a part that saw nothing has maximum -inf, and sums (0, or what a
      // NaN score left) that still count
      const float a = m == -INFINITY ? 1.0f : ex2_mufu(m - top);
      l *= a;
      x.x *= a; x.y *= a; x.z *= a; x.w *= a;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float wk = mk[b] == -INFINITY ? 1.0f : ex2_mufu(mk[b] - top);
        l += lk[b] * wk;
        x.x += y[b].x * wk; x.y += y[b].y * wk; x.z += y[b].z * wk; x.w += y[b].w * wk;
      }
      m = top;
    }
    __syncthreads();  // the segment before has been read
    sx[grp][at] = x;
    sml[grp][at] = make_float2(m, l);
    __syncthreads();
    if (grp != 0) continue;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) top = fmaxf(top, sml[k][at].x);
    float sum = 0.0f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float2 ml = sml[k][at];
      const float4 y = sx[k][at];
      const float wk = ml.x == -INFINITY ? 1.0f : ex2_mufu(ml.x - top);
      sum += ml.y * wk;
      x.x += y.x * wk; x.y += y.y * wk; x.z += y.z * wk; x.w += y.w * wk;
    }
    const Seq s = paged_seq<C>(p, info.y, false);
    const int kvh = info.z / s.blocks;
    const int pair = (info.z - kvh * s.blocks) * C::kRows + row;
    const int tok = pair / p.group;
    if (tok >= s.n) continue;
    float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (FP4 && p.c.v_scale) inv *= p.c.v_scale[kvh];
    const size_t to = (static_cast<size_t>(s.row0) + tok) * p.H + kvh * p.group + pair - tok * p.group;
    *reinterpret_cast<uint2*>(p.o + to * D + d0) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (d0 == 0) p.lse[to] = sum == 0.0f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
  }
}

template <int D, bool FP4, int TILES>
cudaError_t launch_dp(const FwdPagedParams& p, long long max_units, cudaStream_t stream) {
  using C = PagedCfg<D, FP4, TILES>;
  static_assert(C::kWorkers <= kPagedWorkersPerSm && C::kRows <= kPagedRows, "the workspace's shape");
  cudaError_t err = configure_kernel<fa_fwd_paged_kernel<D, FP4, TILES>>(C::kSmemBytes);
  if (err != cudaSuccess) return err;
  const int ctas = sm_count() * C::kCtas;
  if (ctas <= 0) return cudaErrorInvalidConfiguration;
  const int grid = static_cast<int>(max_units < ctas ? max_units : ctas);
  err = launch_dependent(fa_fwd_paged_kernel<D, FP4, TILES>, dim3(static_cast<unsigned int>(grid)),
                         dim3(32 * C::kWarps), C::kSmemBytes, stream, p);
  if (err != cudaSuccess) return err;
  err = launched(1);
  if (err != cudaSuccess) return err;
  const int workers = grid * C::kWarps;
  err = launch_dependent(fa_fwd_paged_join_kernel<D, FP4, TILES>,
                         dim3(static_cast<unsigned int>((workers + kJoinWorkers - 1) / kJoinWorkers), D / 32),
                         dim3(kJoinThreads), 0, stream, p, workers);
  if (err != cudaSuccess) return err;
  return launched(1);
}

template <int D, bool FP4>
cudaError_t launch_d(const FwdPagedParams& p, long long max_units, cudaStream_t stream) {
  // one tile of 8 pairs holds a block where no sequence has more
  return static_cast<long long>(p.max_new) * p.group <= 8 ? launch_dp<D, FP4, 1>(p, max_units, stream)
                                                          : launch_dp<D, FP4, 2>(p, max_units, stream);
}

}  // namespace

int fwd_paged_workers() { return sm_count() * kPagedWorkersPerSm; }

cudaError_t launch_fwd_paged(const FwdPagedParams& p, int d, bool fp4, long long max_units,
                             cudaStream_t stream) {
  if (d == 128) return fp4 ? launch_d<128, true>(p, max_units, stream) : launch_d<128, false>(p, max_units, stream);
  return fp4 ? launch_d<64, true>(p, max_units, stream) : launch_d<64, false>(p, max_units, stream);
}

}  // namespace fa
