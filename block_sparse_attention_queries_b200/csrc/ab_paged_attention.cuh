// Attention of one new token per sequence over a paged key-value cache, for
// every key or for the keys of listed pages.
//
//   O[s, h] = sum_k e^{x_k} v_k / sum_k e^{x_k},  x_k = q_h . k_k / sqrt(d),
//
// over the keys k of sequence s and h's key/value head (of the listed pages),
// with the running maximum and sum of the softmax in fp32.
//
// Each key and value is read once for the G query heads that share it: 2 G
// products per 2-byte element, far below what the tensor cores need per byte,
// so the bound is memory bandwidth and the design keeps bytes in flight:
//  - the (sequence, key/value head) rows are cut into tiles of 64 keys and the
//    whole list of tiles is divided evenly among persistent CTAs, whatever the
//    lengths (share_work); a row that several CTAs share is joined from their
//    partial results by a second kernel;
//  - one warp brings the tiles into a ring of shared-memory stages by TMA (a
//    page of a head is one box of 2 to 16 KB, found through the block table),
//    running ahead across rows;
//  - four warps take 16 keys of each tile each, with a softmax state of their
//    own, joined once per row.
//
// The G heads are the rows of an m16n8k16 product.  P is used as the sum of two
// bfloat16 numbers, so that its rounding (2^-17) does not show next to the
// output's own: for G <= 8 the upper part fills rows 0-7 of the P V product
// and the lower part rows 8-15, at no cost; for G up to 16 two products run
// per half.  V rows that lie behind the sequence's end are set to zero in
// shared memory, since 0 times what an unwritten page holds may be NaN.
#pragma once

#include "ab_paged.cuh"

namespace ab {

constexpr int kDecThreads = 160;   // four consumer warps, one producer warp
constexpr int kDecTile = 64;       // keys per tile
constexpr int kDecMaxParts = 1024; // CTAs at most
constexpr float kDecLazy = 8.f;    // log2 slack of the reference maximum

// Where CTA c's share starts: the row that holds its first tile (-1: behind
// the end), the tile's place in the row, and the row's tiles.
struct DecMeta {
  int row, off, tiles, pad;
};

struct DecArgs {
  PagedView v;
  const __nv_bfloat16* Q;    // [T, Hq, d]
  const int32_t* idx;        // [S, Hkv, max_pages] or null
  const int32_t* count;      // [S, Hkv]
  __nv_bfloat16* O;          // [S, Hq, d]
  float scale_log2;
  int64_t* total;            // workspace: tiles of all rows
  DecMeta* meta;             // [grid + 1]
  float* part_o;             // [grid, 2, 8 RB, d] unnormalised
  float2* part_ml;           // [grid, 2, 8 RB]
};

template <int D, int RB>
struct DecSmem {
  static constexpr int kRow = D * 2;
  static constexpr int kTileBytes = kDecTile * kRow;  // one of K, V
  static constexpr int kStages = D == 128 ? (RB == 1 ? 6 : 5) : (RB == 1 ? 12 : 10);
  static constexpr int kPitch = D + 8;                // floats; rows of a quad's lanes in different banks
  static constexpr int kOffMerge = kStages * 2 * kTileBytes;
  static constexpr int kMergeBytes = 4 * RB * 8 * kPitch * 4;
  static constexpr int kOffMl = kOffMerge + kMergeBytes;  // 4 warps x 8 RB float2
  static constexpr int kOffMeta = kOffMl + 4 * RB * 8 * 8;  // per stage: valid keys of up to 4 pages
  static constexpr int kOffBar = kOffMeta + kStages * 16;
  static constexpr int kOffMisc = kOffBar + kStages * 16;
  static constexpr int kBytes = kOffMisc + 64;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "more shared memory than a CTA may have");
  static_assert(kOffMerge >= kShareSums * 8, "share_work's sums lie in the stages");
};

template <bool kLists>
struct DecRows {
  // tiles of unit u (a sequence, or a row of the lists), all of its heads
  static __device__ __forceinline__ int row_tiles(const DecArgs& a, int s, int hk) {
    const PagedView& v = a.v;
    if (query_row(v, s) < 0) return 0;
    const int pages = pages_of(v, seq_len(v, s));
    int entries = pages;
    if constexpr (kLists) {
      entries = __ldg(a.count + int64_t(s) * v.Hkv + hk);
      if (entries < 0 || entries > v.max_pages) {
        raise_error(AB_ERR_CAPACITY);
        entries = entries < 0 ? 0 : v.max_pages;
      }
    }
    return (entries * v.page + kDecTile - 1) / kDecTile;
  }
  static __device__ __forceinline__ int unit_tiles(const DecArgs& a, int u) {
    if constexpr (kLists) return row_tiles(a, u / a.v.Hkv, u % a.v.Hkv);
    return row_tiles(a, u, 0) * a.v.Hkv;
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

// Barrier among `threads` threads that tells all of them whether any came with `p`.
__device__ __forceinline__ bool bar_any(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}

// D: head dim.  RB: blocks of 8 query heads per key/value head (1: G <= 8,
// 2: G <= 16).  kLists: the pages of a list instead of all.
template <int D, int RB, bool kLists>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const DecArgs a) {
  using SM = DecSmem<D, RB>;
  constexpr int kStages = SM::kStages;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int k) { return sbase + SM::kOffBar + 16u * uint32_t(k); };
  auto empty = [&](int k) { return sbase + SM::kOffBar + 16u * uint32_t(k) + 8u; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::kOffMisc);
  Share* share_out = reinterpret_cast<Share*>(smem + SM::kOffMisc + 16);
  // the prefix sums' scratch: stage memory that no copy has been issued into yet
  int64_t* sums = reinterpret_cast<int64_t*>(smem);
  const PagedView& v = a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      mbar_init(full(k), 1);
      mbar_init(empty(k), 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  const int n_units = kLists ? v.S * v.Hkv : v.S;
  const Share sh = share_work([&](int u) { return DecRows<kLists>::unit_tiles(a, u); }, n_units, blockIdx.x, gridDim.x,
                              sums, share_out);
  fence_proxy_async_smem();  // the scratch's generic accesses come before the copies into it
  __syncthreads();

  // start of the share, for the joining kernel
  int s = kLists ? sh.unit / v.Hkv : sh.unit, hk = kLists ? sh.unit % v.Hkv : 0, off = sh.off;
  if (sh.begin < sh.total) {
    const int T = DecRows<kLists>::row_tiles(a, s, hk);
    if (!kLists) {
      hk = off / T;
      off -= hk * T;
    }
    if (threadIdx.x == 0) a.meta[blockIdx.x] = DecMeta{s * v.Hkv + hk, off, T, 0};
  } else if (threadIdx.x == 0) {
    a.meta[blockIdx.x] = DecMeta{-1, 0, 0, 0};
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.total = sh.total;

  // rows without keys: O = 0
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    if (DecRows<kLists>::unit_tiles(a, u) == 0 && query_row(v, kLists ? u / v.Hkv : u) >= 0) {
      const int n = v.G * D * (kLists ? 1 : v.Hkv);
      uint32_t* o = reinterpret_cast<uint32_t*>(a.O + int64_t(u) * n);
      for (int k = threadIdx.x; k < n / 2; k += kDecThreads) o[k] = 0u;
    }
  }

  // next row with tiles (called by whole warps)
  auto next_row = [&]() -> bool {
    if (!kLists && ++hk < v.Hkv) return true;
    const int u = next_unit([&](int k) { return DecRows<kLists>::unit_tiles(a, k); }, n_units,
                            kLists ? s * v.Hkv + hk + 1 : s + 1);
    s = kLists ? u / v.Hkv : u;
    hk = kLists ? u % v.Hkv : 0;
    return u < n_units;
  };

  int left = sh.n;
  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int per_tile = kDecTile >> v.page_shift;  // list entries of a tile
    const uint32_t page_bytes = uint32_t(SM::kRow) << v.page_shift;
    uint32_t use = 0;  // tiles issued
    bool ok = true;
    while (left > 0 && ok) {
      const int T = DecRows<kLists>::row_tiles(a, s, hk);
      const int n = min(left, T - off);
      const int len = seq_len(v, s), pages = pages_of(v, len);
      const int64_t row = int64_t(s) * v.Hkv + hk;
      const int e_end = kLists ? min(__ldg(a.count + row), v.max_pages) : pages;
      // entries in groups of 32, each lane one: page id (-1: none) and valid keys
      auto fetch = [&](int e, int& id, int& valid) {
        id = -1;
        valid = 0;
        if (e < e_end) {
          const int j = kLists ? __ldg(a.idx + row * v.max_pages + e) : e;
          if (j >= 0 && j < pages) id = __ldg(v.table + int64_t(s) * v.max_pages + j);
          if (id < 0 || id >= v.num_pages) {
            raise_error(AB_ERR_CAPACITY);
            id = -1;
          } else {
            valid = min(v.page, len - (j << v.page_shift));
          }
        }
      };
      const int e0 = off * per_tile, tiles_per_group = 32 / per_tile;
      int id, valid, id_next, valid_next;
      fetch(e0 + lane, id, valid);
      for (int k0 = 0; k0 < n && ok; k0 += tiles_per_group) {
        fetch(e0 + (k0 + tiles_per_group) * per_tile + lane, id_next, valid_next);
        const int kn = min(tiles_per_group, n - k0);
        for (int k = 0; k < kn; ++k, ++use) {
          const int st = int(use % kStages);
          bool got = true;
          if (lane == 0) got = mbar_wait(empty(st), ((use / kStages) & 1) ^ 1, abort_flag);
          if (!__shfl_sync(0xffffffffu, got ? 1 : 0, 0)) { ok = false; break; }
          const int slot = lane - k * per_tile;  // this lane's entry of the tile
          const bool mine = slot >= 0 && slot < per_tile;
          const uint32_t there = __ballot_sync(0xffffffffu, mine && id >= 0);
          if (mine) reinterpret_cast<int*>(smem + SM::kOffMeta + st * 16)[slot] = id >= 0 ? valid : 0;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full(st), 2u * page_bytes * uint32_t(__popc(there)));
          __syncwarp();
          if (mine && id >= 0) {
            const uint32_t dst = sbase + uint32_t(st) * 2u * SM::kTileBytes + uint32_t(slot) * page_bytes;
            tma_load_5d(dst, &tmK, full(st), 0, 0, 0, 0, id * v.Hkv + hk);
            tma_load_5d(dst + SM::kTileBytes, &tmV, full(st), 0, 0, 0, 0, id * v.Hkv + hk);
          }
        }
        id = id_next;
        valid = valid_next;
      }
      left -= n;
      off = 0;
      if (left > 0 && ok) ok = next_row();
    }
    if (lane == 0) {
      // copies in flight land before shared memory is released, also if the
      // consumers gave up: the last use of each stage
      for (uint32_t k = 0; k < uint32_t(kStages) && k < use; ++k) {
        const uint32_t last = use - 1 - ((use - 1 - k) % kStages);
        mbar_wait_drain(full(int(k)), (last / kStages) & 1);
      }
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int key0 = warp * 16;  // this warp's keys of a tile
    // row addresses of the operand loads within a tile (128-byte swizzle, 8-row
    // groups of kHalves KB): K as stored, V transposed
    const int krow = key0 + ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;
    const int vrow = key0 + (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;
    const uint32_t kbase = uint32_t(krow >> 3) * (kHalves * 1024u) + uint32_t(krow & 7) * 128u;
    const uint32_t vbase = uint32_t(vrow >> 3) * (kHalves * 1024u) + uint32_t(vrow & 7) * 128u;
    float* mrg = reinterpret_cast<float*>(smem + SM::kOffMerge);
    float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl);
    uint32_t use = 0;
    int seg = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const int T = DecRows<kLists>::row_tiles(a, s, hk);
      const int n = min(left, T - off);
      const bool whole = n == T;
      // queries: rows g and g + 8 of the 16 x d operand
      uint32_t q0[D / 16][2], q1[D / 16][2];
      {
        const __nv_bfloat16* q = a.Q + (int64_t(query_row(v, s)) * v.Hkv + hk) * v.G * D + 2 * t;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            q0[k][z] = g < v.G ? __ldg(reinterpret_cast<const uint32_t*>(q + g * D + 16 * k + 8 * z)) : 0u;
            q1[k][z] = RB == 2 && g + 8 < v.G
                           ? __ldg(reinterpret_cast<const uint32_t*>(q + (g + 8) * D + 16 * k + 8 * z))
                           : 0u;
          }
        }
      }
      float o[RB][D / 8][4];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][k][e] = 0.f;
      float m[RB], l[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      for (int k = 0; k < n; ++k, ++use) {
        const int st = int(use % kStages);
        const bool got = mbar_wait(full(st), (use / kStages) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        const int* mt = reinterpret_cast<const int*>(smem + SM::kOffMeta + st * 16);
        const int valid = min(16, mt[key0 >> v.page_shift] - (key0 & (v.page - 1)));
        const uint32_t kt = sbase + uint32_t(st) * 2u * SM::kTileBytes, vt = kt + SM::kTileBytes;
        if (valid > 0) {
          if (valid < 16) {
            // zero the V rows behind the end
            for (int r = key0 + valid; r < key0 + 16; ++r)
              for (int h = 0; h < kHalves; ++h)
                *reinterpret_cast<uint32_t*>(smem + size_t(st) * 2 * SM::kTileBytes + SM::kTileBytes +
                                             (r >> 3) * (kHalves * 1024) + h * 1024 + (r & 7) * 128 + lane * 4) = 0u;
            fence_proxy_async_smem();
            __syncwarp();
          }
          // S = Q K^T for 16 keys: two n-tiles, each in two accumulators
          float c[2][2][4] = {};
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            const int ch = 2 * kk + kch;
            ldmatrix_x4(kt + kbase + uint32_t(ch >> 3) * 1024u + uint32_t(((ch & 7) ^ (krow & 7)) << 4), b);
            mma_16816(c[0][kk & 1], q0[kk][0], q1[kk][0], q0[kk][1], q1[kk][1], b[0], b[1]);
            mma_16816(c[1][kk & 1], q0[kk][0], q1[kk][0], q0[kk][1], q1[kk][1], b[2], b[3]);
          }
          uint32_t hi[RB][4], lo[RB][4];  // P of keys (0-7: 2t, 2t+1), (8-15: 2t, 2t+1) as A operands
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = (e >> 1) * 8 + 2 * t + (e & 1);
              x[e] = c[e >> 1][0][2 * r + (e & 1)] + c[e >> 1][1][2 * r + (e & 1)];
              if (key >= valid) x[e] = -INFINITY;
            }
            float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * a.scale_log2;
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (__any_sync(0xffffffffu, mx > m[r] + kDecLazy)) {
              const float mn = fmaxf(m[r], mx);
              const float al = mn == -INFINITY ? 1.f : ex2_approx(m[r] - mn);
              m[r] = mn;
              l[r] *= al;
#pragma unroll
              for (int k8 = 0; k8 < D / 8; ++k8)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[r][k8][e] *= al;
            }
            const float ref = m[r] == -INFINITY ? 0.f : m[r];
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ex2_approx(fmaf(x[e], a.scale_log2, -ref));
              l[r] += p[e];
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              hi[r][z] = pack_bf16x2(p[2 * z], p[2 * z + 1]);
              lo[r][z] = pack_bf16x2(p[2 * z] - __uint_as_float(hi[r][z] << 16),
                                     p[2 * z + 1] - __uint_as_float(hi[r][z] & 0xFFFF0000u));
            }
          }
          // O += P V: rows 0-7 the upper part of P, rows 8-15 the lower
#pragma unroll
          for (int np = 0; np < D / 16; ++np) {
            uint32_t b[4];
            const int ch = 2 * np + vch;
            ldmatrix_x4_trans(vt + vbase + uint32_t(ch >> 3) * 1024u + uint32_t(((ch & 7) ^ (vrow & 7)) << 4), b);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
              mma_16816(o[r][2 * np], hi[r][0], lo[r][0], hi[r][1], lo[r][1], b[0], b[1]);
              mma_16816(o[r][2 * np + 1], hi[r][0], lo[r][0], hi[r][1], lo[r][1], b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }
      // join the four warps' results of this row (a warp that gave up comes too,
      // and all of them learn of it)
      asm volatile("bar.sync 1, 128;" ::: "memory");  // the buffer's last readers are done
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int head = r * 8 + g;
        if (t == 0) ml[warp * RB * 8 + head] = make_float2(m[r], l[r]);
        float* dst = mrg + (warp * RB * 8 + head) * SM::kPitch + 2 * t;
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          *reinterpret_cast<float2*>(dst + 8 * k) = make_float2(o[r][k][0] + o[r][k][2], o[r][k][1] + o[r][k][3]);
      }
      ok = !bar_any(1, 128, !ok);
      if (!ok) break;
      const int64_t row = int64_t(s) * v.Hkv + hk;
      const int slot = seg == 0 ? 0 : 1;  // a partial row is this CTA's first or its last
      for (int e = threadIdx.x * 2; e < v.G * D; e += 256) {
        const int head = e / D, i = e % D;
        float2 z[4];
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          z[w] = ml[w * RB * 8 + head];
          mm = fmaxf(mm, z[w].x);
        }
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = ex2_approx(z[w].x - ref);
          const float2 ow = *reinterpret_cast<const float2*>(mrg + (w * RB * 8 + head) * SM::kPitch + i);
          ll += z[w].y * f;
          o0 += ow.x * f;
          o1 += ow.y * f;
        }
        if (whole) {
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
          *reinterpret_cast<uint32_t*>(a.O + (row * v.G + head) * D + i) = pack_bf16x2(o0 * inv, o1 * inv);
        } else {
          const int64_t at = (int64_t(blockIdx.x) * 2 + slot) * (RB * 8) + head;
          *reinterpret_cast<float2*>(a.part_o + at * D + i) = make_float2(o0, o1);
          if (i == 0) a.part_ml[at] = make_float2(mm, ll);
        }
      }
      ++seg;
      left -= n;
      off = 0;
      if (left > 0) ok = next_row();
    }
  }
}

// Joins the partial results of the rows that several CTAs share.  Block
// (c, h) takes the row that CTA c's share starts inside of, if CTA c - 1's
// share holds the row's first tile; one thread per output value and group of
// parts.
constexpr int kJoinGroups = 4;

template <int D>
__global__ void __launch_bounds__(D * kJoinGroups)
    paged_join_kernel(const DecArgs a, int C, int heads_pad) {
  __shared__ float so[kJoinGroups][D], sl[kJoinGroups], sm[kJoinGroups];
  const int c = blockIdx.x + 1, h = blockIdx.y;
  const DecMeta mt = a.meta[c];
  if (mt.row < 0 || mt.off == 0) return;
  const int64_t total = *a.total;
  auto begin = [&](int k) { return total * k / C; };
  const int64_t start = begin(c) - mt.off, end = start + mt.tiles;  // the row's tiles
  if (begin(c - 1) > start) return;
  int last = c;  // last CTA with a tile of the row
  while (last + 1 < C && begin(last + 1) < end) ++last;
  const int grp = threadIdx.x / D, i = threadIdx.x % D;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k = c - 1 + grp; k <= last; k += kJoinGroups) {
    if (begin(k + 1) == begin(k)) continue;  // a CTA without work
    const int slot = k == c - 1 && begin(k) != start ? 1 : 0;
    const int64_t at = (int64_t(k) * 2 + slot) * heads_pad + h;
    const float2 z = a.part_ml[at];
    const float x = a.part_o[at * D + i];
    const float mm = fmaxf(m, z.x);
    if (mm != -INFINITY) {
      const float fa = ex2_approx(m - mm), fb = ex2_approx(z.x - mm);
      l = l * fa + z.y * fb;
      o = o * fa + x * fb;
      m = mm;
    }
  }
  so[grp][i] = o;
  if (i == 0) {
    sl[grp] = l;
    sm[grp] = m;
  }
  __syncthreads();
  if (grp == 0) {
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < kJoinGroups; ++k) mm = fmaxf(mm, sm[k]);
    float ll = 0.f, oo = 0.f;
    if (mm != -INFINITY) {
#pragma unroll
      for (int k = 0; k < kJoinGroups; ++k) {
        const float f = ex2_approx(sm[k] - mm);
        ll += sl[k] * f;
        oo += so[k][i] * f;
      }
    }
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
    a.O[(int64_t(mt.row) * a.v.G + h) * D + i] = __float2bfloat16(oo * inv);
  }
}

}  // namespace ab
