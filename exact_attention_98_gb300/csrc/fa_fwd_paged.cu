// Attention of each sequence's last tokens over its paged key/value cache.
//
// The token at position p of a sequence sees the cached positions j <= p with
// p - j < window, and the first `sinks` positions: S_j = scale q.k_j over
// these, O = softmax(S) V, LSE = ln sum exp S_j.
//
// Bound by HBM: each visible cached row is read once per key head and serves
// every query head of the group, so the rows of the matrix products are
// (token, head of the group), 16 of them at a time: products this narrow are
// far below the tensor cores' rate, and mma.sync (whose operands come from
// registers, where a 4-bit row is turned into halves anyway) carries them.
//
// Work: a segment is (sequence, key head, block of 16 rows) and a list of
// 64-position tiles: those of the first tokens, then those of the window.
// All tiles of all segments are laid out in one line, which the CTAs cut
// into equal pieces, whatever the lengths of the sequences (read on the
// device, so that a captured graph serves any lengths).  A CTA that holds
// the whole of a segment writes its rows; the parts of a segment that
// several CTAs share go to the workspace (at most two parts per CTA), and a
// second kernel joins them by their maxima and sums.
//
// A CTA: four warps of 16 positions of each tile, each with its own running
// maxima, sums and accumulators (joined at the end of a segment), and a
// fifth that copies the tiles' pages into a ring of stages in shared memory:
// bf16 by tiled TMA with the 128-byte swizzle that ldmatrix reads without
// conflicts, 4-bit blocks as plain bulk copies, codes and scales together.
//
// 4 bits: codes become halves exactly (e2m1 x e4m3 has six bits), so the only
// roundings are those of P to fp16 and of the result.  Q is scaled to fp16
// by a power of two per row.  The products are free to permute d: lane
// (g, c) of a warp reads of key g the codes [c d/4, (c+1) d/4) in one load,
// and of the keys 2c, 2c+1 (V) the codes [g d/8, (g+1) d/8).
#include <limits.h>

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kTileKeys = 64;
constexpr int kRows = 16;         // rows of a segment
constexpr int kWarps = 4;         // compute warps
constexpr int kFwdThreads = 160;  // and the one that loads
constexpr int kCtasPerSm = 2;

enum : unsigned int {
  kSitePagedFull = 0x511,
  kSitePagedEmpty = 0x512,
};

// Rows and sums keep a maximum that is at most this much (log2 units) below
// the true one, so that accumulators are rescaled rarely.  bf16 keeps the
// dominant weight near 1 (its rounding error reaches O); fp16's spacing is 8
// times finer and its range holds 2^8 with room below.
template <bool FP4>
__device__ constexpr float kSlack = FP4 ? 8.0f : 2.0f;

template <int D, bool FP4>
struct PagedCfg {
  static constexpr int kStageBytes = FP4 ? 2 * kTileKeys * (D / 2 + D / 16) : 2 * kTileKeys * D * 2;
  static constexpr int kStages = FP4 ? (D == 128 ? 8 : 12) : (D == 128 ? 3 : 5);
  static constexpr int kJoinOff = kStages * kStageBytes;  // [4 warps][16 rows][32] fp32
  static constexpr int kJoinBytes = kWarps * kRows * 32 * 4;
  static constexpr int kStatOff = kJoinOff + kJoinBytes;  // [4 warps][2][16]: maxima, sums
  static constexpr int kBarOff = kStatOff + kWarps * 2 * kRows * 4;
  static constexpr int kAbortOff = kBarOff + 2 * kStages * 8;
  static constexpr int kScanOff = kAbortOff + 16;  // long long [8] for the scan
  static constexpr int kSmemBytes = kScanOff + 8 * 8 + 1024;
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
};

// What a sequence asks for.
struct Seq {
  int row0, n;      // its rows of q
  int len;          // cached positions
  int first_tiles;  // tiles of the first tokens
  int win_tile;     // the window's first tile
  int tiles;        // units of a segment: its tiles, or 1 without any
  int loads;        // its tiles
  int blocks;       // blocks of 16 rows
};

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
  if (s.len < 0 || s.len > most) {
    if (report) record_status(p.status, kStatusInvalid, kSitePagedLength);
    s.len = s.len < 0 ? 0 : static_cast<int>(most);
  }
  s.len = max(0, s.len - extra);
  const int p0 = max(0, s.len - s.n);
  const int lo = p.window == INT_MAX ? 0 : max(0, p0 - p.window + 1);
  const int end = (s.len + kTileKeys - 1) / kTileKeys;
  s.win_tile = lo / kTileKeys;
  s.first_tiles = min((min(p.sinks, s.len) + kTileKeys - 1) / kTileKeys, s.win_tile);
  s.loads = s.n > 0 ? s.first_tiles + end - s.win_tile : 0;
  s.tiles = max(1, s.loads);
  s.blocks = (s.n * p.group + kRows - 1) / kRows;
  return s;
}

__device__ __forceinline__ long long seq_units(const FwdPagedParams& p, const Seq& s) {
  return static_cast<long long>(s.tiles) * s.blocks * p.c.Hkv;
}

// A CTA's place in the line of units.
struct Walk {
  long long left;  // units left to this CTA
  int b;           // sequence
  Seq s;
  int seg;         // key head * blocks + block of rows
  int tile;        // first unit within the segment
};

// Moves to the next segment after `done` units of this one.
__device__ __forceinline__ void walk_next(const FwdPagedParams& p, Walk& w, int done) {
  w.left -= done;
  w.tile = 0;
  if (++w.seg < w.s.blocks * p.c.Hkv) return;
  w.seg = 0;
  while (w.left > 0 && w.b + 1 < p.c.B) {
    w.s = paged_seq(p, ++w.b, false);
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Untiled bulk copy global -> shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <int D, bool FP4>
__global__ void __launch_bounds__(kFwdThreads, kCtasPerSm)
    fa_fwd_paged_kernel(const __grid_constant__ FwdPagedParams p) {
  using C = PagedCfg<D, FP4>;
  constexpr int kSteps = D / 16;    // k16 steps of Q K^T
  constexpr int kNTiles = D / 8;    // n8 tiles of P V
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);
  const WaitCtl ctl{abort_flag, p.status};
  auto full = [&](int s) -> uint32_t { return sbase + C::kBarOff + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return sbase + C::kBarOff + 8u * (C::kStages + s); };
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  __syncthreads();

  // ---- this CTA's piece of the line of units
  long long* scan = reinterpret_cast<long long*>(smem + C::kScanOff);
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
    for (int w = 0; w < kFwdThreads / 32; ++w) {
      if (w < warp) v += scan[w];
      total += scan[w];
    }
    return v;
  };
  long long total = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += kFwdThreads) {
    const int b = b0 + threadIdx.x;
    long long t;
    block_scan(b < p.c.B ? seq_units(p, paged_seq(p, b, blockIdx.x == 0)) : 0, t);
    total += t;
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  if (blockIdx.x >= ctas) {
    if (threadIdx.x == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  auto piece = [&](long long c) { return total / ctas * c + min(c, total % ctas); };
  const long long u0 = piece(blockIdx.x);
  long long before = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += kFwdThreads) {
    const int b = b0 + threadIdx.x;
    const long long mine = b < p.c.B ? seq_units(p, paged_seq(p, b, false)) : 0;
    long long t;
    const long long end = before + block_scan(mine, t);
    if (u0 < end && u0 >= end - mine) {
      scan[6] = b;
      scan[7] = u0 - (end - mine);
    }
    before += t;
    if (u0 < before) break;  // the same for every thread
  }
  __syncthreads();
  Walk w;
  w.left = piece(blockIdx.x + 1) - u0;
  w.b = static_cast<int>(scan[6]);
  w.s = paged_seq(p, w.b, false);
  w.seg = static_cast<int>(scan[7] / w.s.tiles);
  w.tile = static_cast<int>(scan[7] % w.s.tiles);

  const int sub_keys = min(1 << p.c.page_shift, kTileKeys);  // positions that one copy brings
  const int sub_shift = min(p.c.page_shift, 6);
  const int subs = kTileKeys >> sub_shift;  // copies of a tile

  if (warp == kWarps) {
    // ---------------------------------------------------------------- loads
    int used = 0;
    bool ok = true;
    while (w.left > 0 && ok) {
      const int kvh = w.seg / w.s.blocks;
      const int t1 = static_cast<int>(min(static_cast<long long>(w.s.tiles), w.tile + w.left));
      const int n_load = min(t1, w.s.loads);
      const int* table = p.c.page_table + static_cast<size_t>(w.b) * p.c.max_pages;
      const int batch = 32 >> (6 - sub_shift);  // tiles whose page numbers one load by the warp brings
      int ids = -1;  // lane: page of tile (lane / subs) of the batch, part lane % subs
      for (int i = w.tile; i < n_load; ++i) {
        const int in_batch = (i - w.tile) % batch;
        auto tile_of = [&](int u) { return u < w.s.first_tiles ? u : u - w.s.first_tiles + w.s.win_tile; };
        if (in_batch == 0) {
          const int u = i + lane / subs;
          const int key = tile_of(u) * kTileKeys + (lane % subs) * sub_keys;
          ids = -1;  // behind the sequence: not loaded
          if (u < n_load && key < w.s.len) {
            ids = table[key >> p.c.page_shift];
            if (ids < 0 || ids >= p.c.num_pages) {
              record_status(p.status, kStatusInvalid, kSitePagedPage);
              ids = -1;
            }
          }
        }
        const int stage = used % C::kStages;
        const int use = used / C::kStages;
        if (use > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(empty(stage), (use - 1) & 1, ctl, kSitePagedEmpty));
          if (!ok) break;
        }
        const uint32_t dst = sbase + stage * C::kStageBytes;
        const int tile = tile_of(i);
        // the page that this lane copies
        int mine = __shfl_sync(0xffffffffu, ids, in_batch * subs + (lane % subs));
        if (lane >= subs) mine = -1;
        const unsigned int live = __ballot_sync(0xffffffffu, mine >= 0);
        const uint32_t sub_bytes = C::kStageBytes >> (6 - sub_shift);
        if (lane == 0) mbar_arrive_expect_tx(full(stage), __popc(live) * sub_bytes);
        __syncwarp();
        if (mine >= 0) {
          const size_t block = static_cast<size_t>(mine) * p.c.Hkv + kvh;
          // 128-position pages: the tile is one half of the page
          const int in_page = p.c.page_shift > 6 ? (tile * kTileKeys) & ((1 << p.c.page_shift) - 1) : 0;
          if constexpr (FP4) {
            const size_t half = paged_half_bytes(true, 1 << p.c.page_shift, D);
            const uint8_t* from = p.c.pages + block * 2 * half;
            const uint32_t to = dst + lane * sub_bytes;
            if (p.c.page_shift <= 6) {
              bulk_load(to, from, sub_bytes, full(stage));
            } else {
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                const uint8_t* f = from + kv * half;
                const uint32_t t = to + kv * (sub_bytes / 2);
                bulk_load(t, f + static_cast<size_t>(in_page) * (D / 2), kTileKeys * (D / 2), full(stage));
                bulk_load(t + kTileKeys * (D / 2),
                          f + (static_cast<size_t>(D / 2) << p.c.page_shift) + in_page * (D / 16),
                          kTileKeys * (D / 16), full(stage));
              }
            }
          } else {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(dst + (kv * (D / 64) + h) * (kTileKeys * 128) + lane * sub_keys * 128, &p.tm,
                            full(stage), h * 64, in_page, static_cast<int>(block * 2 + kv));
          }
        }
        __syncwarp();
        ++used;
      }
      walk_next(p, w, t1 - w.tile);
    }
    // every copy lands before shared memory is released (waits only on the
    // give-up path)
    if (!ok)
      for (int u = max(0, used - C::kStages); u < used; ++u)
        mbar_wait_drain(full(u % C::kStages), (u / C::kStages) & 1);
    return;
  }

  // ------------------------------------------------------------------ compute
  const int g = lane >> 2, c = lane & 3;
  float* join = reinterpret_cast<float*>(smem + C::kJoinOff);
  float* stat = reinterpret_cast<float*>(smem + C::kStatOff);
  int used = 0;
  if (threadIdx.x == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
  while (w.left > 0) {
    const int kvh = w.seg / w.s.blocks;
    const int block = w.seg - kvh * w.s.blocks;
    const int t1 = static_cast<int>(min(static_cast<long long>(w.s.tiles), w.tile + w.left));
    const int n_load = min(t1, w.s.loads);
    // rows g and g + 8 of the block: their token, head and position
    int row_at[2], pos[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = block * kRows + g + 8 * r;
      const int tok = row / p.group;
      const bool in = tok < w.s.n;
      row_at[r] = in ? tok : -1;
      pos[r] = in ? w.s.len - w.s.n + tok : -1;
    }
    const int last_row = min(w.s.n * p.group, (block + 1) * kRows) - 1;
    const int p_lo = w.s.len - w.s.n + (block * kRows) / p.group;  // the rows' positions: least and most
    const int p_hi = w.s.len - w.s.n + last_row / p.group;

    // Q as the products' A operand
    uint32_t qa[kSteps][4];
    float mul[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int head = kvh * p.group + (block * kRows + g + 8 * r) % p.group;
      const __nv_bfloat16* src =
          p.q + (w.s.row0 + static_cast<long long>(max(row_at[r], 0))) * p.q_row + head * p.q_head;
      mul[r] = p.scale;
      if constexpr (FP4) {
        // d = c D/4 + 4 s + {0, 1} (a0) and + {2, 3} (a2)
        uint4 raw[D / 32];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row_at[r] >= 0) raw[i] = *reinterpret_cast<const uint4*>(src + c * (D / 4) + 8 * i);
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[e] << 16)),
                                     fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // a power of two brings the row's largest magnitude into [1, 2):
        // down is 2^-e, up its inverse (kept in the normal range)
        const int e = min(253, max(1, static_cast<int>((__float_as_uint(amax) >> 23) & 255u)));
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        mul[r] *= __uint_as_float(static_cast<uint32_t>(e) << 23);
        if (p.c.k_scale) mul[r] *= p.c.k_scale[kvh];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2)
            qa[2 * i + (e2 >> 1)][(e2 & 1) * 2 + r] =
                pack_f16x2(__uint_as_float(x[e2] << 16) * down, __uint_as_float(x[e2] & 0xFFFF0000u) * down);
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            uint32_t x = 0u;
            if (row_at[r] >= 0) x = *reinterpret_cast<const uint32_t*>(src + s * 16 + k8 * 8 + 2 * c);
            qa[s][k8 * 2 + r] = x;
          }
      }
    }

    float acc[kNTiles][4];
#pragma unroll
    for (int j = 0; j < kNTiles; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY};  // running maxima, log2 units
    float l[2] = {0.0f, 0.0f};            // this lane's share of the sums

    for (int i = w.tile; i < n_load; ++i, ++used) {
      const int tile = i < w.s.first_tiles ? i : i - w.s.first_tiles + w.s.win_tile;
      const int key0 = tile * kTileKeys + warp * 16;  // this warp's 16 positions
      const int stage = used % C::kStages;
      mbar_wait(full(stage), (used / C::kStages) & 1, ctl, kSitePagedFull);
      __syncwarp();
      const uint8_t* st = smem + stage * C::kStageBytes;
      const uint32_t st_s = sbase + stage * C::kStageBytes;
      // every position visible to every row?
      const bool edge = key0 + 15 > p_lo || (static_cast<long long>(key0) <= static_cast<long long>(p_hi) - p.window &&
                                             key0 + 16 > p.sinks);
      // 4 bits: the sub-block that holds this warp's positions
      const int sub = (warp * 16) >> sub_shift;
      const int in_sub = (warp * 16) & (sub_keys - 1);
      const uint8_t* kblk = st + sub * (C::kStageBytes >> (6 - sub_shift));
      const uint8_t* vblk = kblk + (C::kStageBytes >> (7 - sub_shift));

      // S = Q K^T: position key0 + 8 nt + 2c + {0, 1} of rows g (0, 1), g + 8 (2, 3)
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
      if constexpr (FP4) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int key = in_sub + nt * 8 + g;
          uint32_t codes[D / 32];
          const uint8_t* kc = kblk + key * (D / 2) + c * (D / 8);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(kc);
            codes[0] = x.x; codes[1] = x.y; codes[2] = x.z; codes[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kc);
            codes[0] = x.x; codes[1] = x.y;
          }
          const uint8_t* ks = kblk + (D / 2) * sub_keys + key * (D / 16) + c * (D / 64);
          uint32_t sc[D / 64];  // the scales of this lane's 16-element blocks, twice each
#pragma unroll
          for (int k = 0; k < D / 64; ++k) sc[k] = e4m3x2_to_f16x2(ks[k] * 0x101u);
#pragma unroll
          for (int wd = 0; wd < D / 32; ++wd) {
            uint32_t h[4];
            e2m1x8_to_f16x2(codes[wd], h);
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = hmul2(h[k], sc[wd >> 1]);
            mma16816<true>(s[nt], qa[2 * wd], h[0], h[1]);
            mma16816<true>(s[nt], qa[2 * wd + 1], h[2], h[3]);
          }
        }
      } else {
        // lanes 0-7, 8-15: keys 0-7, both halves of 16 elements; 16-31: keys 8-15
        const int row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
        const int hi = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b[4];
          const int chunk = (k & 3) * 2 + hi;
          ldmatrix_x4(st_s + (k >> 2) * (kTileKeys * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), b);
          mma16816<false>(s[0], qa[k], b[0], b[1]);
          mma16816<false>(s[1], qa[k], b[2], b[3]);
        }
      }

      // scaled scores; masked ones -inf
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] *= mul[e >> 1];
          if (edge) {
            const int j = key0 + nt * 8 + 2 * c + (e & 1);
            const int q = pos[e >> 1];
            if (!(j <= q && (static_cast<long long>(q) - j < p.window || j < p.sinks))) s[nt][e] = -INFINITY;
          }
        }
      float mx[2], ref[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      // the reference moves only when it is left behind by more than the slack
      const bool move0 = mx[0] > m[0] + kSlack<FP4>, move1 = mx[1] > m[1] + kSlack<FP4>;
      if (__any_sync(0xffffffffu, move0 || move1)) {
        const float a0 = move0 ? ex2_mufu(m[0] - mx[0]) : 1.0f;
        const float a1 = move1 ? ex2_mufu(m[1] - mx[1]) : 1.0f;
        if (move0) m[0] = mx[0];
        if (move1) m[1] = mx[1];
        l[0] *= a0;
        l[1] *= a1;
#pragma unroll
        for (int j = 0; j < kNTiles; ++j) {
          acc[j][0] *= a0;
          acc[j][1] *= a0;
          acc[j][2] *= a1;
          acc[j][3] *= a1;
        }
      }
      ref[0] = m[0] == -INFINITY ? 0.0f : m[0];
      ref[1] = m[1] == -INFINITY ? 0.0f : m[1];
      uint32_t pa[4];  // P as the A operand: (row g, nt 0), (g + 8, nt 0), (g, nt 1), (g + 8, nt 1)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = ex2_mufu(s[nt][2 * r] - ref[r]), y = ex2_mufu(s[nt][2 * r + 1] - ref[r]);
          l[r] += x + y;
          pa[nt * 2 + r] = FP4 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
        }

      // O += P V.  A position that no row sees has weight 0, but its row of V
      // may hold anything (the rest of a page, infinities): it is zeroed.
      // Bit 2 nt + e: position key0 + 8 nt + 2c + e.
      unsigned int keep = 15u;
      if (edge) {
        keep = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = key0 + (k >> 1) * 8 + 2 * c + (k & 1);
          const bool seen = j <= p_hi && (j < p.sinks || static_cast<long long>(p_lo) - j < p.window);
          keep |= seen ? 1u << k : 0u;
        }
      }
      if constexpr (FP4) {
        // n-tile j of lane g is d = g D/8 + j
        uint32_t sc[2];  // scales of the keys' pairs
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint8_t* vs = vblk + (D / 2) * sub_keys + (in_sub + nt * 8 + 2 * c) * (D / 16) + (g * D) / 128;
          const uint32_t lo = (keep >> (2 * nt)) & 1u ? vs[0] : 0u;
          const uint32_t hi = (keep >> (2 * nt + 1)) & 1u ? vs[D / 16] : 0u;
          sc[nt] = e4m3x2_to_f16x2(lo | (hi << 8));
        }
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          uint32_t even[2][4], odd[2][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint8_t* vc = vblk + (in_sub + nt * 8 + 2 * c) * (D / 2) + g * (D / 16) + wd * 4;
            const uint32_t a = *reinterpret_cast<const uint32_t*>(vc);
            const uint32_t b = *reinterpret_cast<const uint32_t*>(vc + D / 2);
            // byte i: element 2i (or 2i+1) of key 2c low, of key 2c+1 high
            e2m1x8_to_f16x2((a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4), even[nt]);
            e2m1x8_to_f16x2(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), odd[nt]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              even[nt][k] = hmul2(even[nt][k], sc[nt]);
              odd[nt][k] = hmul2(odd[nt][k], sc[nt]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma16816<true>(acc[wd * 8 + 2 * k], pa, even[0][k], even[1][k]);
            mma16816<true>(acc[wd * 8 + 2 * k + 1], pa, odd[0][k], odd[1][k]);
          }
        }
      } else {
        // lanes 0-7: keys 0-7 of columns 8j..; 8-15: keys 8-15; 16-31: the next 8 columns
        const int row = warp * 16 + (lane & 15);
        const int hi = lane >> 4;
        const uint32_t k01 = ((keep & 1u) ? 0xFFFFu : 0u) | ((keep & 2u) ? 0xFFFF0000u : 0u);
        const uint32_t k23 = ((keep & 4u) ? 0xFFFFu : 0u) | ((keep & 8u) ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int j = 0; j < kNTiles; j += 2) {
          uint32_t b[4];
          const int chunk = (j & 7) + hi;
          ldmatrix_x4_t(st_s + (D / 64 + (j >> 3)) * (kTileKeys * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), b);
          if (edge) {
            b[0] &= k01; b[1] &= k23; b[2] &= k01; b[3] &= k23;
          }
          mma16816<false>(acc[j], pa, b[0], b[1]);
          mma16816<false>(acc[j + 1], pa, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(stage));
    }

    // ---- the four warps' parts of the rows joined
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        stat[(warp * 2) * kRows + g + 8 * r] = m[r];
        stat[(warp * 2 + 1) * kRows + g + 8 * r] = l[r];
      }
    }
    named_bar_sync(1, 32 * kWarps);
    float weight[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stat[(k * 2) * kRows + g + 8 * r]);
      weight[r] = m[r] == -INFINITY ? 0.0f : ex2_mufu(m[r] - top);
    }
    // thread: 4 of 32 columns of a row, round by round
    const int jr = threadIdx.x >> 3, jc = threadIdx.x & 7;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stat[(k * 2) * kRows + jr]);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float mk = stat[(k * 2) * kRows + jr];
      if (mk != -INFINITY) sum += stat[(k * 2 + 1) * kRows + jr] * ex2_mufu(mk - top);
    }
    const bool whole = w.tile == 0 && t1 == w.s.tiles;
    const int out_row = block * kRows + jr;
    const int tok = out_row / p.group;
    const bool in = tok < w.s.n;
    const int head = kvh * p.group + out_row - tok * p.group;
    const size_t at = (static_cast<size_t>(w.s.row0) + tok) * p.H + head;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (w.tile == 0 ? 1 : 0);
    float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    if (FP4 && p.c.v_scale) inv *= p.c.v_scale[kvh];
#pragma unroll
    for (int round = 0; round < kNTiles / 4; ++round) {
      if (round > 0) named_bar_sync(1, 32 * kWarps);
#pragma unroll
      for (int j4 = 0; j4 < 4; ++j4)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = FP4 ? (2 * c + (e & 1)) * 4 + j4 : j4 * 8 + 2 * c + (e & 1);
          join[(warp * kRows + g + 8 * (e >> 1)) * 32 + col] = acc[round * 4 + j4][e] * weight[e >> 1];
        }
      named_bar_sync(1, 32 * kWarps);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(join + (k * kRows + jr) * 32 + jc * 4);
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      const int d0 = FP4 ? jc * (D / 8) + round * 4 : round * 32 + jc * 4;
      if (!whole) {
        *reinterpret_cast<float4*>(p.part_o + (slot * kRows + jr) * D + d0) = x;
      } else if (in) {
        *reinterpret_cast<uint2*>(p.o + at * D + d0) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
      }
    }
    if (jc == 0) {
      if (!whole) {
        p.part_ml[slot * 2 * kRows + jr] = top;
        p.part_ml[slot * 2 * kRows + kRows + jr] = sum;
      } else if (in) {
        p.lse[at] = sum == 0.0f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
      }
    }
    if (threadIdx.x == 0 && w.tile == 0 && !whole) {
      // the segment goes on in the CTAs after this one: how many
      const long long rest = w.s.tiles - t1;
      int parts = 1;
      for (long long c2 = static_cast<long long>(blockIdx.x) + 1, got = 0; got < rest; ++c2, ++parts)
        got += piece(c2 + 1) - piece(c2);
      p.info[blockIdx.x] = make_int4(parts, w.b, w.seg, 0);
    }
    named_bar_sync(1, 32 * kWarps);  // stat and join are free again
    walk_next(p, w, t1 - w.tile);
  }
}

// Joins the parts of the segment that starts in CTA blockIdx.x and goes on in
// the CTAs after it: the first part is that CTA's second slot, the others the
// following CTAs' first ones.  A thread takes 4 columns of a row.
template <int D, bool FP4>
__global__ void __launch_bounds__(kRows * D / 4)
    fa_fwd_paged_join_kernel(const __grid_constant__ FwdPagedParams p) {
  grid_dependency_wait();
  const int4 info = p.info[blockIdx.x];
  if (info.x == 0) return;
  const Seq s = paged_seq(p, info.y, false);
  const int kvh = info.z / s.blocks;
  const int block = info.z - kvh * s.blocks;
  const int row = threadIdx.x / (D / 4);
  const int d0 = (threadIdx.x % (D / 4)) * 4;
  const int out_row = block * kRows + row;
  const int tok = out_row / p.group;
  if (tok >= s.n) return;
  auto slot = [&](int k) {
    return 2 * (static_cast<size_t>(blockIdx.x) + k) + (k == 0 ? 1 : 0);
  };
  float top = -INFINITY;
  for (int k = 0; k < info.x; ++k) top = fmaxf(top, p.part_ml[slot(k) * 2 * kRows + row]);
  float sum = 0.0f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < info.x; ++k) {
    const float mk = p.part_ml[slot(k) * 2 * kRows + row];
    const float lk = p.part_ml[slot(k) * 2 * kRows + kRows + row];
    const float4 y = *reinterpret_cast<const float4*>(p.part_o + (slot(k) * kRows + row) * D + d0);
    const float wk = mk == -INFINITY ? 0.0f : ex2_mufu(mk - top);
    sum += lk * wk;
    x.x += y.x * wk; x.y += y.y * wk; x.z += y.z * wk; x.w += y.w * wk;
  }
  float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  if (FP4 && p.c.v_scale) inv *= p.c.v_scale[kvh];
  const size_t at = (static_cast<size_t>(s.row0) + tok) * p.H + kvh * p.group + out_row - tok * p.group;
  *reinterpret_cast<uint2*>(p.o + at * D + d0) =
      make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  if (d0 == 0) p.lse[at] = sum == 0.0f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
}

template <int D, bool FP4>
cudaError_t launch_dp(const FwdPagedParams& p, long long max_units, cudaStream_t stream) {
  using C = PagedCfg<D, FP4>;
  cudaError_t err = cudaFuncSetAttribute(fa_fwd_paged_kernel<D, FP4>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  const int ctas = fwd_paged_ctas();
  if (ctas <= 0) return cudaErrorInvalidConfiguration;
  const unsigned int grid = static_cast<unsigned int>(max_units < ctas ? max_units : ctas);
  err = launch_dependent(fa_fwd_paged_kernel<D, FP4>, dim3(grid), dim3(kFwdThreads), C::kSmemBytes, stream, p);
  if (err != cudaSuccess) return err;
  err = launched(1);
  if (err != cudaSuccess) return err;
  err = launch_dependent(fa_fwd_paged_join_kernel<D, FP4>, dim3(grid), dim3(kRows * D / 4), 0, stream, p);
  if (err != cudaSuccess) return err;
  return launched(1);
}

}  // namespace

int fwd_paged_ctas() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms * kCtasPerSm;
}

cudaError_t launch_fwd_paged(const FwdPagedParams& p, int d, bool fp4, long long max_units,
                             cudaStream_t stream) {
  if (d == 128) return fp4 ? launch_dp<128, true>(p, max_units, stream) : launch_dp<128, false>(p, max_units, stream);
  return fp4 ? launch_dp<64, true>(p, max_units, stream) : launch_dp<64, false>(p, max_units, stream);
}

}  // namespace fa
