// Attention of one new token per sequence over a paged key-value cache, for
// every key or for the keys of listed pages.
//
//   O[s, h] = sum_k e^{x_k} v_k / sum_k e^{x_k},  x_k = q_h . k_k / sqrt(d),
//
// over the keys k of sequence s and h's key/value head (of the listed pages),
// with the running maximum and sums of the softmax in fp32.
//
// Each key and value is read once for the G query heads that share it: 2 G
// products per 2-byte element, far below what the tensor cores need per byte,
// so the bound is memory bandwidth and the design keeps bytes in flight:
//  - the (sequence, key/value head) rows are cut into tiles of 64 keys (128 for
//    d = 64) and the whole list of tiles is divided evenly among persistent
//    CTAs, whatever the lengths (share_work; a row's start and end count as half
//    a tile); a row that several CTAs share is joined from their partial results
//    by a second kernel (short tables: rows stay whole);
//  - one warp plans 32 tiles at a time, a lane for each: the tile's row, its
//    pages through the lists and the block table.  All lookups of 32 tiles run
//    side by side, so that rows of a single tile cost no more than long ones;
//  - three warps bring the planned tiles into a ring of shared-memory stages, 16
//    bytes a lane and copy, only the rows that hold keys, and the row's queries
//    where a row begins.  (By TMA a tile of four 4 KB boxes each of K and V took
//    1000 cycles, one of 2 KB boxes about as long: at most 32 bytes a cycle and
//    about 100 cycles a box, where HBM needs 23 bytes a cycle.)
//  - two groups of four warps take the rows in turn, so that one row's start and
//    end, about 2000 cycles, overlap the next one's tiles (for G > 8 each group
//    takes its half of the heads of every row); a group's warps take 16 (32)
//    keys of each tile each, with a softmax state of their own, joined once per
//    row.
//
// The products are m16n8k16 (one in 8 cycles a quarter of an SM, measured), so
// their number counts where 16 heads share a key: S is taken transposed, 16 keys
// by 8 heads, and P turned back on its way into P V (heads by dims), a quarter
// fewer products than with the heads as rows throughout (359 us against 314).
//
// P is used as the sum of two bfloat16 numbers, so that its rounding (2^-17)
// does not show next to the output's own: a group has at most 8 heads, so the
// upper part fills rows 0-7 of the P V product and the lower part rows 8-15, at
// no cost.  (An infinite value times a lower part is not what it is times the whole:
// join_parts.)  V rows that lie behind the sequence's end are set to zero in the
// operand, since 0 times what an unwritten page holds may be NaN.
//
// Fewer bits than fp32 elsewhere: exponentials by ex2.approx (2^-22, as in the
// selection and the joins), and the accumulators of the products, which cut off
// (kDecOwnSum).
//
// Measured: 8 sequences of 122 thousand keys, 4 key heads of 8 query heads, 295 us
// (6.8 TB/s of keys and values; 16 query heads each 300), 64 sequences of 1 to
// 16384 keys 72 us (5.8 TB/s), one of 777 keys 9.2 us with the join.
#pragma once

#include <type_traits>

#include "ab_norm_rope.cuh"
#include "ab_paged.cuh"

namespace ab {

// two groups of four consumer warps, three warps that copy, the planning warp
constexpr int kDecGroups = 2;
constexpr int kDecThreads = kDecGroups * 128 + 128;
// Keys per tile: 32 KB of keys and values (d = 64 with tiles of 64 keys: 40 heads,
// 11 % of 30 thousand keys kept, 83 us against 67).
__host__ __device__ constexpr int dec_tile(int D) { return D == 128 ? 64 : 128; }
// A row's start and end, in halves of a tile: 64 sequences of 1 to 16384 keys 72.6
// us, 79.6 with 0; 512 of 1 to 600 keys 57, with 0 67, with 2 64.
constexpr int kDecRowCost = 1;
// Tables of at most this many tiles: no row is divided, so that there is nothing to
// join.  12 heads of 128, 256 keys 7.9 us, divided and joined 8.2, 128 keys 6.5 and
// 8.1; but 384 keys 9.2 and 8.5; 64 sequences of 2 heads of 64, 512 keys 10.0 and 10.8.
constexpr int kWholeTiles = 4;
constexpr int kDecMaxParts = 1024; // CTAs at most
constexpr float kDecLazy = 8.f;    // log2 slack of the reference maximum
// Tiles of a row whose P V stays in the products' own accumulators.  Their sum cuts
// off what does not fit, to one side, so its error grows with its length (2000
// tiles of random values in one CTA: small outputs 3 % off); behind these many tiles
// it is taken out and added in fp32, to nearest, in shared memory.  8 sequences of
// 122 thousand keys 295 us, 293 without, with 16 query heads a key head 302 and 295;
// by 16 tiles 298 and 308; every tile's product added in registers 298 and 338.
constexpr int kDecOwnSum = 64;

// A CTA's share, for the joining kernel: its tiles [begin, begin + n) of the
// list, and the row that begins in it and ends behind it (-1: none), that row's
// end in the list, and which of the CTA's two parts it is.
struct DecMeta {
  int begin, n, row, end, slot, pad[3];
};

// A planned tile.
struct DecTile {
  int coord[8];  // page * Hkv + head of up to 8 pages, -1: none
  int valid[2];  // valid keys of each, a byte each
  int row;       // s * Hkv + key/value head
  int qrow;      // row of Q
  int flags;
  int pad[3];
};
// of the CTA's tiles of a row: the first, the last; of the row: the first, the last;
// every kDecOwnSum-th, one behind such a one; shift: rows begun before
enum : int { kTileFirst = 1, kTileLast = 2, kRowStart = 4, kRowEnd = 8, kTileOut = 16, kTileMore = 32, kTileRow = 6 };

struct DecArgs {
  PagedView v;
  const __nv_bfloat16 *Q, *K, *V;  // [T, Hq, d], [num_pages, Hkv, page, d]
  const int32_t* idx;        // [S, Hkv, max_pages] or null
  const int32_t* count;      // [S, Hkv]
  __nv_bfloat16* O;          // [S, Hq, d]
  float scale_log2;
  bool whole;                // no row is divided
  DecMeta* meta;             // workspace: [grid]
  float* part_o;             // [grid, 2, 8 or 16 heads, d] unnormalised
  float2* part_ml;           // [grid, 2, 8 or 16 heads]
};

template <int D>
struct DecSmem {
  static constexpr int kRow = D * 2;
  static constexpr int kTile = dec_tile(D);
  static constexpr int kTileBytes = kTile * kRow;     // one of K, V
  static constexpr int kStages = 5;
  static constexpr int kPitch = D + 8;                // floats; rows of a quad's lanes in different banks
  static constexpr int kQPitch = kRow + 16;           // bytes, for the same reason
  static constexpr int kQBytes = kMaxGroup * kQPitch;
  static constexpr int kOffQ = kStages * 2 * kTileBytes;
  static constexpr int kOffMerge = kOffQ + kStages * kQBytes;
  static constexpr int kMergeBytes = 4 * 8 * kPitch * 4;
  static constexpr int kOffMl = kOffMerge + kDecGroups * kMergeBytes;  // per group: 4 warps x 8 float2
  static constexpr int kMlBytes = 4 * 8 * 8;
  static constexpr int kOffPlan = kOffMl + kDecGroups * kMlBytes;      // 2 x 32 planned tiles
  static constexpr int kOffMeta = kOffPlan + 2 * 32 * int(sizeof(DecTile));  // per stage: valid, row, flags
  static constexpr int kOffBar = kOffMeta + kStages * 16;
  static constexpr int kNumBars = 2 * kStages + 4 + kDecGroups;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "more shared memory than a CTA may have");
  static_assert(kOffQ >= kShareSums * 8, "share_work's sums lie in the stages");
};

template <int D, bool kLists>
struct DecRows {
  // list entries (pages) of a row
  static __device__ __forceinline__ int row_entries(const DecArgs& a, int s, int hk) {
    const PagedView& v = a.v;
    if (query_row(v, s) < 0) return 0;
    if constexpr (kLists) {
      const int n = __ldg(a.count + int64_t(s) * v.Hkv + hk);
      if (n < 0 || n > v.max_pages) {
        raise_error(AB_ERR_CAPACITY);
        return n < 0 ? 0 : v.max_pages;
      }
      return n;
    }
    return pages_of(v, seq_len(v, s));
  }
  static __device__ __forceinline__ int tiles_of(const DecArgs& a, int entries) {
    return ((entries << a.v.page_shift) + dec_tile(D) - 1) / dec_tile(D);
  }
  // unit u: a row of the lists, or a sequence with all of its heads
  static __device__ __forceinline__ UnitWork work(const DecArgs& a, int u) {
    if constexpr (kLists) return {1, tiles_of(a, row_entries(a, u / a.v.Hkv, u % a.v.Hkv))};
    return {a.v.Hkv, tiles_of(a, row_entries(a, u, 0))};
  }
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Arrive on `bar` when all of this thread's cp.async copies so far have landed
// (counted among the barrier's arrivals).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Transpose of an 8 x 8 matrix of 16-bit values, two in a row per lane.
__device__ __forceinline__ uint32_t turn_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The sums of both parts of P.  Where a value is infinite the upper one is infinite
// or NaN, as it should be, and the lower one, of weights that are negative or zero, is
// not looked at.
__device__ __forceinline__ float join_parts(float upper, float lower) {
  return fabsf(upper) < INFINITY ? upper + lower : upper;
}

// As lane0_wait, and what the other side wrote before its arrival is seen by every
// lane (a shuffle orders no memory).
__device__ __forceinline__ bool lead_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = lane0_wait(bar, parity, abort_flag);
  __syncwarp();
  return ok;
}

// D: head dim.  kLists: the pages of a list instead of all.
template <int D, bool kLists>
__global__ void __launch_bounds__(kDecThreads, 1) paged_attention_kernel(const __grid_constant__ DecArgs a) {
  using SM = DecSmem<D>;
  using Rows = DecRows<D, kLists>;
  constexpr int kStages = SM::kStages;
  constexpr int kHalves = D / 64;
  constexpr int kCopyWarp = 4 * kDecGroups, kPlanWarp = kCopyWarp + 3;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int k) { return sbase + SM::kOffBar + 16u * uint32_t(k); };
  auto empty = [&](int k) { return sbase + SM::kOffBar + 16u * uint32_t(k) + 8u; };
  auto plan_full = [&](int k) { return full(kStages + k); };
  auto plan_empty = [&](int k) { return empty(kStages + k); };
  auto join_bar = [&](int k) { return full(kStages + 2) + 8u * uint32_t(k); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::kOffMisc);
  DecTile* plan = reinterpret_cast<DecTile*>(smem + SM::kOffPlan);
  // the prefix sums' scratch: stage memory that no copy has been issued into yet
  int2* sums = reinterpret_cast<int2*>(smem);
  const PagedView& v = a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      mbar_init(full(k), 97);  // the copies of three warps' lanes, and the tile's description
      mbar_init(empty(k), 4 * kDecGroups);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(plan_full(k), 1);
      mbar_init(plan_empty(k), 3);
    }
    for (int k = 0; k < kDecGroups; ++k) mbar_init(join_bar(k), 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  const int n_units = kLists ? v.S * v.Hkv : v.S;
  const Share sh =
      share_work([&](int u) { return Rows::work(a, u); }, kDecRowCost, a.whole, n_units, blockIdx.x, gridDim.x, sums);
  __syncthreads();  // the scratch has been read

  if (warp == kPlanWarp) {
    // ------------------------------------------------------------ planner
    constexpr int kMaxPages = SM::kTile / 16;
    const int per_tile = SM::kTile >> v.page_shift;  // pages of a tile
    DecMeta meta{sh.begin, sh.n, -1, 0, 0, {0, 0, 0}};
    if (lane == 0) a.meta[blockIdx.x] = meta;  // what the joining kernel finds if a wait below gives up
    __syncwarp();
    int unit = sh.unit, pos = sh.off;  // tile `base` of the share is tile `pos` from the start of unit `unit` on
    int rows = 0;  // rows begun
    bool ok = true;
    for (int base = 0, batch = 0; base < sh.n && ok; base += 32, ++batch) {
      // find this lane's tile: the unit, and the tile's place in it
      int x = pos + lane, mine = -1;
      bool open = base + lane < sh.n;
      for (int u0 = unit; __any_sync(0xffffffffu, open) && u0 < n_units; u0 += 32) {
        const UnitWork w = u0 + lane < n_units ? Rows::work(a, u0 + lane) : UnitWork{0, 0};
        const int t = w.rows * w.tiles;
        const int incl = warp_inclusive(t), all = __shfl_sync(0xffffffffu, incl, 31);
        int l = 0;  // first unit of these 32 whose sum passes x
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(0xffffffffu, incl, l + o - 1) <= x) l += o;
        const int before = __shfl_sync(0xffffffffu, incl - t, l);
        if (open) {
          if (x < all) {
            mine = u0 + l;
            x -= before;
            open = false;
          } else {
            x -= all;
          }
        }
      }
      DecTile d{};
#pragma unroll
      for (int k = 0; k < 8; ++k) d.coord[k] = -1;
      if (mine >= 0) {
        int s = mine, hk = 0, off = x;
        if constexpr (kLists) {
          s = mine / v.Hkv;
          hk = mine - s * v.Hkv;
        }
        const int entries = Rows::row_entries(a, s, hk), T = Rows::tiles_of(a, entries);
        if constexpr (!kLists) {
          hk = off / T;
          off -= hk * T;
        }
        const int64_t row = int64_t(s) * v.Hkv + hk;
        const int len = seq_len(v, s), pages = pages_of(v, len), at = base + lane;
        d.row = int(row);
        d.qrow = query_row(v, s);
        d.flags = (off == 0 || at == 0 ? kTileFirst : 0) | (off == T - 1 || at == sh.n - 1 ? kTileLast : 0) |
                  (off == 0 ? kRowStart : 0) | (off == T - 1 ? kRowEnd : 0) |
                  (min(off, at) % kDecOwnSum == kDecOwnSum - 1 ? kTileOut : 0) | (min(off, at) >= kDecOwnSum ? kTileMore : 0);
        if (at == sh.n - 1) {
          if (off < T - 1 && off <= at) {  // the row begins here and goes on behind the share
            meta.row = d.row;
            meta.end = sh.begin + at - off + T;
            meta.slot = off == at ? 0 : 1;
          }
          a.meta[blockIdx.x] = meta;
        }
        int j[kMaxPages], id[kMaxPages];
#pragma unroll
        for (int k = 0; k < kMaxPages; ++k) {
          const int e = off * per_tile + k;
          j[k] = -1;
          if (k < per_tile && e < entries) j[k] = kLists ? __ldg(a.idx + row * v.max_pages + e) : e;
        }
#pragma unroll
        for (int k = 0; k < kMaxPages; ++k) {
          id[k] = -1;
          if (j[k] >= 0 && j[k] < pages) id[k] = __ldg(v.table + int64_t(s) * v.max_pages + j[k]);
        }
#pragma unroll
        for (int k = 0; k < kMaxPages; ++k) {
          if (k < per_tile && off * per_tile + k < entries) {
            if (id[k] < 0 || id[k] >= v.num_pages) {
              raise_error(AB_ERR_CAPACITY);
            } else {
              d.coord[k] = id[k] * v.Hkv + hk;
              d.valid[k >> 2] |= min(v.page, len - (j[k] << v.page_shift)) << (8 * (k & 3));
            }
          }
        }
      }
      const uint32_t firsts = __ballot_sync(0xffffffffu, d.flags & kTileFirst);
      d.flags |= (rows + __popc(firsts & (0xffffffffu >> (31 - lane))) - 1) << kTileRow;
      rows += __popc(firsts);
      ok = lead_wait(plan_empty(batch & 1), ((batch >> 1) & 1) ^ 1, abort_flag);
      if (!ok) break;
      plan[(batch & 1) * 32 + lane] = d;
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_full(batch & 1));
      // the next batch begins behind lane 31's tile
      unit = __shfl_sync(0xffffffffu, mine, 31);
      pos = __shfl_sync(0xffffffffu, x, 31) + 1;
      if (unit < 0) break;  // the share's last batch
    }
  } else if (warp >= kCopyWarp) {
    // -------------------------------------------------------------- copies
    // The 16-key pieces of a tile's K and V are dealt out to the three warps;
    // a lane copies 16 bytes at a time into their place in the 128-byte swizzle.
    constexpr int kCols = D / 8;          // 16-byte columns of a row
    constexpr int kStep = 32 / kCols;     // rows that a warp copies at once
    const int mine = warp - kCopyWarp;
    const int col = lane % kCols, row0 = lane / kCols;
    uint32_t use = 0;  // tiles issued
    bool ok = true;
    for (int base = 0, batch = 0; base < sh.n && ok; base += 32, ++batch) {
      ok = lead_wait(plan_full(batch & 1), (batch >> 1) & 1, abort_flag);
      const int n = min(32, sh.n - base);
      for (int k = 0; k < n && ok; ++k, ++use) {
        const DecTile* d = plan + (batch & 1) * 32 + k;
        const int st = int(use % kStages);
        ok = lead_wait(empty(st), ((use / kStages) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const int flags = d->flags;
        const uint64_t valid = uint64_t(uint32_t(d->valid[0])) | uint64_t(uint32_t(d->valid[1])) << 32;
        constexpr int kPieces = SM::kTile / 16;  // of K, and as many of V
#pragma unroll
        for (int x = 0; x < (2 * kPieces + 2) / 3; ++x) {
          const int piece = mine + 3 * x;
          const bool of_k = piece < kPieces;
          const int key0 = (piece & (kPieces - 1)) * 16, entry = key0 >> v.page_shift, in_page = key0 & (v.page - 1);
          const int rows = min(16, int(uint32_t(valid >> (8 * entry)) & 255u) - in_page);
          if (piece < 2 * kPieces && rows > 0) {
            const __nv_bfloat16* src =
                (of_k ? a.K : a.V) + (int64_t(d->coord[entry]) * v.page + in_page + row0) * D + col * 8;
            const uint32_t dst = sbase + uint32_t(st) * 2u * SM::kTileBytes + (of_k ? 0u : uint32_t(SM::kTileBytes)) +
                                 uint32_t(key0 >> 3) * (kHalves * 1024u) + uint32_t(col >> 3) * 1024u;
#pragma unroll
            for (int r = 0; r < 16; r += kStep) {
              const int row = r + row0;
              if (row < rows)
                cp_async16(dst + uint32_t(row >> 3) * (kHalves * 1024u) + uint32_t(row & 7) * 128u +
                               (uint32_t((col & 7) ^ (row & 7)) << 4),
                           src + r * D);
            }
          }
        }
        if (mine == 2 && (flags & kTileFirst)) {
          const int hk = d->row % v.Hkv;
          const __nv_bfloat16* q = a.Q + ((int64_t(d->qrow) * v.Hkv + hk) * v.G + row0) * D + col * 8;
          const uint32_t dst = sbase + SM::kOffQ + uint32_t(st * SM::kQBytes + row0 * SM::kQPitch + col * 16);
          for (int h = row0; h < v.G; h += kStep, q += kStep * D)
            cp_async16(dst + uint32_t((h - row0) * SM::kQPitch), q);
        }
        if (mine == 0 && lane == 0) {
          *reinterpret_cast<int4*>(smem + SM::kOffMeta + st * 16) = make_int4(d->valid[0], d->valid[1], d->row, flags);
          mbar_arrive(full(st));  // the copies' arrival below orders no plain store
        }
        cp_async_arrive(full(st));  // arrives when this lane's copies have landed
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty(batch & 1));
    }
    cp_async_wait<0>();
  } else {
    // ----------------------------------------------------------- consumers
    // units without keys: O = 0 (a lane looks at one, the warp writes)
    for (int64_t k0 = int64_t(warp) * 32; blockIdx.x + k0 * gridDim.x < n_units; k0 += 128 * kDecGroups) {
      const int64_t u = blockIdx.x + (k0 + lane) * gridDim.x;
      const bool none = u < n_units && Rows::work(a, int(u)).tiles == 0 && query_row(v, kLists ? int(u) / v.Hkv : int(u)) >= 0;
      for (uint32_t some = __ballot_sync(0xffffffffu, none); some; some &= some - 1) {
        const int n = v.G * D * (kLists ? 1 : v.Hkv);
        uint32_t* z = reinterpret_cast<uint32_t*>(a.O + (blockIdx.x + (k0 + __ffs(some) - 1) * gridDim.x) * n);
        for (int k = lane; k < n / 2; k += 32) z[k] = 0u;
      }
    }
    const int g = lane >> 2, t = lane & 3;
    const int group = warp >> 2, gwarp = warp & 3, gthread = threadIdx.x & 127;
    // this warp's keys of a tile: 16 of every 64.  Row addresses of the operand
    // loads (128-byte swizzle, 8-row groups of kHalves KB): K as stored, V
    // transposed, both by the same addresses
    constexpr int NB = SM::kTile / 64;
    constexpr uint32_t kBlock = 8 * kHalves * 1024;  // 64 keys
    // 16 rows of a warp: lanes 0-15 the first 16-byte column of a pair, 16-31 the second
    const int lrow = gwarp * 16 + (lane & 15);
    // column 2 k + (lane >> 4) of a row is at (base + row) ^ (k << 5)
    const uint32_t lbase = uint32_t(lrow >> 3) * (kHalves * 1024u) + uint32_t(lrow & 7) * 128u +
                           uint32_t(((lane >> 4) ^ (lrow & 7)) << 4);
    float* mrg = reinterpret_cast<float*>(smem + SM::kOffMerge + group * SM::kMergeBytes);
    float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl + group * SM::kMlBytes);
    bool started = false;  // the current row's first tile is this CTA's
    const bool split = v.G > 8;
    const int head0 = split ? group * 8 : 0, heads = min(8, v.G - head0);  // this group's
    uint32_t q[D / 16][2];  // queries: the d x 8 operand
    float o[D / 8][4];      // head g and dims 8 k + 2 t, + 1: upper and lower part of P
    float m[2], l[2];       // of heads 2 t, 2 t + 1 (l: this lane's keys)
    // all of the group's warps are here (bounded like every wait: one of them may have given up)
    uint32_t joins = 0;
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(join_bar(group));
      return warp_wait(join_bar(group), joins++ & 1, abort_flag);
    };
    for (uint32_t use = 0; use < uint32_t(sh.n); ++use) {
      const int st = int(use % kStages);
      const bool got = mbar_wait(full(st), (use / kStages) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, got)) break;
      const int4 mt = *reinterpret_cast<const int4*>(smem + SM::kOffMeta + st * 16);
      const int flags = mt.w;
      if (!split && ((flags >> kTileRow) & 1) != group) {  // another group's row
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
        continue;
      }
      if (flags & kTileFirst) {
        const uint8_t* from = smem + SM::kOffQ + st * SM::kQBytes + (head0 + g) * SM::kQPitch + 4 * t;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
#pragma unroll
          for (int z = 0; z < 2; ++z) q[k][z] = g < heads ? *reinterpret_cast<const uint32_t*>(from + 32 * k + 16 * z) : 0u;
        }
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
        started = flags & kRowStart;
      }
      const uint64_t valid8 = uint64_t(uint32_t(mt.x)) | uint64_t(uint32_t(mt.y)) << 32;
      int valid[NB];  // keys of each 16
      bool some = false, all = true;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int key = nb * 64 + gwarp * 16;
        valid[nb] = int(uint32_t(valid8 >> (8 * (key >> v.page_shift))) & 255u) - (key & (v.page - 1));
        some = some || valid[nb] > 0;
        all = all && valid[nb] >= 16;
      }
      const uint32_t kt = sbase + uint32_t(st) * 2u * SM::kTileBytes, vt = kt + SM::kTileBytes;
      if (some) {
        // S^T = K Q^T, 16 keys by 8 heads, each in two accumulators
        float c[NB][2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            uint32_t k[4];
            ldmatrix_x4(((kt + lbase) ^ uint32_t((kk & 3) << 5)) + nb * kBlock + uint32_t(kk >> 2) * 1024u, k);
            mma_16816(c[nb][kk & 1], k[0], k[1], k[2], k[3], q[kk][0], q[kk][1]);
          }
        }
        float x[NB][4];  // key g, heads 2 t and 2 t + 1; key g + 8, the same heads
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[nb][e] = c[nb][0][e] + c[nb][1][e];
            if (!all && (e >> 1) * 8 + g >= valid[nb]) x[nb][e] = -INFINITY;
            mx[e & 1] = fmaxf(mx[e & 1], x[nb][e]);
          }
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
          for (int z = 0; z < 2; ++z) mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], off));
        mx[0] *= a.scale_log2;
        mx[1] *= a.scale_log2;
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kDecLazy || mx[1] > m[1] + kDecLazy)) {
          float al[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float mn = fmaxf(m[z], mx[z]);
            al[z] = mn == -INFINITY ? 1.f : ex2_approx(m[z] - mn);
            m[z] = mn;
            l[z] *= al[z];
          }
          const float a0 = __shfl_sync(0xffffffffu, al[0], g >> 1), a1 = __shfl_sync(0xffffffffu, al[1], g >> 1);
          const float of_g = g & 1 ? a1 : a0;
#pragma unroll
          for (int k8 = 0; k8 < D / 8; ++k8)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k8][e] *= of_g;
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        uint32_t hi[NB][2], lo[NB][2];  // P of head g, keys (0-7: 2t, 2t+1), (8-15: 2t, 2t+1), as A operands
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float p0 = ex2_approx(fmaf(x[nb][2 * z], a.scale_log2, -ref[0]));
            const float p1 = ex2_approx(fmaf(x[nb][2 * z + 1], a.scale_log2, -ref[1]));
            l[0] += p0;
            l[1] += p1;
            const uint32_t up = pack_bf16x2(p0, p1);
            hi[nb][z] = turn_8x8(up);
            lo[nb][z] = turn_8x8(pack_bf16x2(p0 - __uint_as_float(up << 16), p1 - __uint_as_float(up & 0xFFFF0000u)));
          }
        }
        // O += P V: rows 0-7 the upper part of P, rows 8-15 the lower; V rows
        // behind the end count as zero
        auto add_pv = [&](auto partial) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            uint32_t keep[2];
#pragma unroll
            for (int z = 0; z < 2; ++z)
              keep[z] = (z * 8 + 2 * t < valid[nb] ? 0xFFFFu : 0u) | (z * 8 + 2 * t + 1 < valid[nb] ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int np = 0; np < D / 16; ++np) {
              uint32_t b[4];
              ldmatrix_x4_trans(((vt + lbase) ^ uint32_t((np & 3) << 5)) + nb * kBlock + uint32_t(np >> 2) * 1024u, b);
              if constexpr (decltype(partial)::value) {
                b[0] &= keep[0];
                b[1] &= keep[1];
                b[2] &= keep[0];
                b[3] &= keep[1];
              }
              mma_16816(o[2 * np], hi[nb][0], lo[nb][0], hi[nb][1], lo[nb][1], b[0], b[1]);
              mma_16816(o[2 * np + 1], hi[nb][0], lo[nb][0], hi[nb][1], lo[nb][1], b[2], b[3]);
            }
          }
        };
        if (all) add_pv(std::false_type{});
        else add_pv(std::true_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
      if (!(flags & (kTileLast | kTileOut))) continue;

      // what the accumulators hold goes to this lane's places in the group's buffer
      if (flags & kTileMore) {  // with what is there, in terms of the maximum now
        const float m0 = __shfl_sync(0xffffffffu, m[0], g >> 1), m1 = __shfl_sync(0xffffffffu, m[1], g >> 1);
        const float m_g = g & 1 ? m1 : m0;
        const float f = m_g == -INFINITY ? 0.f : ex2_approx(ml[gwarp * 8 + g].x - m_g);
        const float* src = mrg + (gwarp * 8 + g) * SM::kPitch + 2 * t;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const float2 x = *reinterpret_cast<const float2*>(src + 8 * k);
          o[k][0] = fmaf(x.x, f, o[k][0]);
          o[k][1] = fmaf(x.y, f, o[k][1]);
        }
        __syncwarp();
      } else if (!group_sync()) {  // its last readers are done
        break;
      }
      float lsum[2] = {l[0], l[1]};
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int z = 0; z < 2; ++z) lsum[z] += __shfl_xor_sync(0xffffffffu, lsum[z], off);
      if (g == 0) {
        ml[gwarp * 8 + 2 * t] = make_float2(m[0], lsum[0]);
        ml[gwarp * 8 + 2 * t + 1] = make_float2(m[1], lsum[1]);
      }
      float* dst = mrg + (gwarp * 8 + g) * SM::kPitch + 2 * t;
#pragma unroll
      for (int k = 0; k < D / 8; ++k)
        *reinterpret_cast<float2*>(dst + 8 * k) = make_float2(join_parts(o[k][0], o[k][2]), join_parts(o[k][1], o[k][3]));
      if (!(flags & kTileLast)) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
        continue;
      }

      // join the four warps' results of this row
      if (!group_sync()) break;
      const bool whole = started && (flags & kRowEnd);
      const int64_t row = mt.z;
      const int slot = flags >> kTileRow == 0 ? 0 : 1;  // a partial row is this CTA's first or its last
      for (int e = gthread * 4; e < heads * D; e += 512) {
        const int head = e / D, i = e % D;
        float2 z[4];
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          z[w] = ml[w * 8 + head];
          mm = fmaxf(mm, z[w].x);
        }
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = ex2_approx(z[w].x - ref);
          const float4 ow = *reinterpret_cast<const float4*>(mrg + (w * 8 + head) * SM::kPitch + i);
          ll += z[w].y * f;
          s4.x += ow.x * f;
          s4.y += ow.y * f;
          s4.z += ow.z * f;
          s4.w += ow.w * f;
        }
        if (whole) {
          const float inv = ll == 0.f ? 0.f : 1.f / ll;  // NaN stays NaN
          *reinterpret_cast<uint2*>(a.O + (row * v.G + head0 + head) * D + i) =
              make_uint2(pack_bf16x2(s4.x * inv, s4.y * inv), pack_bf16x2(s4.z * inv, s4.w * inv));
        } else {
          const int64_t at = (int64_t(blockIdx.x) * 2 + slot) * (split ? 16 : 8) + head0 + head;
          *reinterpret_cast<float4*>(a.part_o + at * D + i) = s4;
          if (i == 0) a.part_ml[at] = make_float2(mm, ll);
        }
      }
    }
  }
}

// Joins the partial results of the rows that several CTAs share.  Block (c, h)
// takes head h of the row that begins in CTA c's share and ends behind it; eight
// warps take every eighth part, four values a lane.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const __grid_constant__ DecArgs a, int C, int heads_pad) {
  constexpr int kVec = D / 32;
  __shared__ float so[kJoinWarps][D];
  __shared__ float2 sml[kJoinWarps];
  pdl_wait();
  const int c = blockIdx.x, h = blockIdx.y;
  const DecMeta mt = a.meta[c];
  if (mt.row < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, o[kVec] = {};
  for (int k = c + warp; k < C; k += kJoinWarps) {
    const int2 share = *reinterpret_cast<const int2*>(a.meta + k);
    if (share.x >= mt.end) break;
    if (share.y == 0) continue;
    const int64_t at = (int64_t(k) * 2 + (k == c ? mt.slot : 0)) * heads_pad + h;
    const float2 z = a.part_ml[at];
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const float2 y = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * kVec + i);
      x[i] = y.x;
      x[i + 1] = y.y;
    }
    const float mm = fmaxf(m, z.x), ref = mm == -INFINITY ? 0.f : mm;
    const float fa = ex2_approx(m - ref), fb = ex2_approx(z.x - ref);
    l = l * fa + z.y * fb;
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = o[i] * fa + x[i] * fb;
    m = mm;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) so[warp][lane * kVec + i] = o[i];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mm = -INFINITY;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) mm = fmaxf(mm, sml[k].x);
  const float ref = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f, oo = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    const float f = ex2_approx(sml[k].x - ref);
    ll += sml[k].y * f;
    oo += so[k][threadIdx.x] * f;
  }
  a.O[(int64_t(mt.row) * a.v.G + h) * D + threadIdx.x] = __float2bfloat16(ll == 0.f ? 0.f : oo / ll);
}

}  // namespace ab
