// A paged key-value cache: block tables and slot maps from the requests'
// lengths, page summaries, and the selection of pages for one new token per
// sequence.  The attention over the cache is in ab_paged_attention.cuh.
//
// The cache holds num_pages pages of `page` tokens; K and V are
// [num_pages, Hkv, page, d], so that one page of one head is a contiguous run
// of 2 to 16 KB.  Sequence s's j-th page is table[s][j]; slot = page id * page
// + offset names a token's place.
#pragma once

#include <climits>

#include "ab_norm_rope.cuh"
#include "ab_ptx.cuh"

namespace ab {

constexpr int kMaxSeqs = 8192;   // sequences of a block table: their prefix sums fit in shared memory
constexpr int kMaxGroup = 16;    // query heads per key/value head

struct PagedView {
  const int32_t* table;   // [S, max_pages]
  const int32_t* lens;    // [S]
  const int32_t* cu_new;  // [S + 1] or null: row of Q (null: row s)
  int T;                  // rows of Q
  int S, Hkv, G;
  int page, page_shift, num_pages, max_pages;
};

// Tokens of sequence s, 0 if the length is out of range.
__device__ __forceinline__ int seq_len(const PagedView& v, int s) {
  const int n = __ldg(v.lens + s);
  if (n < 0 || n > v.max_pages << v.page_shift) {
    raise_error(AB_ERR_CAPACITY);
    return 0;
  }
  return n;
}
__device__ __forceinline__ int pages_of(const PagedView& v, int tokens) {
  return (tokens + v.page - 1) >> v.page_shift;
}
// Row of Q that holds sequence s's newest token, -1 if it has none.
__device__ __forceinline__ int query_row(const PagedView& v, int s) {
  if (!v.cu_new) return s;
  const int lo = __ldg(v.cu_new + s), hi = __ldg(v.cu_new + s + 1);
  if (hi <= lo) return -1;
  if (hi > v.T || lo < 0) {
    raise_error(AB_ERR_CAPACITY);
    return -1;
  }
  return hi - 1;
}

// ------------------------------------------------------------------- plan
// One cluster of 8 CTAs.  Each CTA computes the prefix sums of all sequences
// in shared memory (the inputs are a few KB), then the CTAs share the list
// entries, table entries and slots.  The cluster's barrier stands between the
// last read of lens and free_count and their update, so both may be updated in
// place.  Bound by latency: a step of 256 sequences moves a few KB and takes
// 6.8 us, a single token's 4.4.
constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;

struct PlanArgs {
  int S, T, page, page_shift, num_pages, max_pages;
  const int32_t *n_new, *lens;
  int32_t* lens_out;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t *cu_new, *slots, *positions;
};

// Counts that stop at 2^31 - 1 (more than any list or slot map holds).
struct PlanScan {
  uint32_t rel, need, want;
};
__device__ __forceinline__ PlanScan operator+(const PlanScan& a, const PlanScan& b) {
  constexpr uint32_t kMost = 0x7FFFFFFFu;
  return {min(a.rel + b.rel, kMost), min(a.need + b.need, kMost), min(a.want + b.want, kMost)};
}
__device__ __forceinline__ PlanScan shfl_up(const PlanScan& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.rel, o), __shfl_up_sync(0xffffffffu, a.need, o),
          __shfl_up_sync(0xffffffffu, a.want, o)};
}
__device__ __forceinline__ PlanScan shfl_at(const PlanScan& a, int l) {
  return {__shfl_sync(0xffffffffu, a.rel, l), __shfl_sync(0xffffffffu, a.need, l), __shfl_sync(0xffffffffu, a.want, l)};
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  // prefix sums over the sequences ([0] = 0) and the lengths before the step
  int32_t* cu_want = plan_smem;                 // [S + 1]
  int32_t* cu_need = cu_want + a.S + 1;         // [S + 1]
  int32_t* cu_rel = cu_need + a.S + 1;          // [S + 1]
  int32_t* old_len = cu_rel + a.S + 1;          // [S]
  __shared__ PlanScan warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();

  int F0 = *a.free_count;
  if (F0 < 0 || F0 > a.num_pages) {
    if (tid == 0) raise_error(AB_ERR_CAPACITY);
    F0 = F0 < 0 ? 0 : a.num_pages;
  }

  // what sequence s gives back and asks for
  auto ask = [&](int s) -> PlanScan {
    PlanScan v{0, 0, 0};
    if (s >= a.S) return v;
    int len = a.lens[s];
    const int n = a.n_new[s];
    const int cap = a.max_pages << a.page_shift;
    bool bad = n < -1;
    if (len < 0 || len > cap) {
      bad = true;
      len = len < 0 ? 0 : cap;
    }
    old_len[s] = len;
    const int old = (len + a.page - 1) >> a.page_shift;
    if (!bad && n == -1) {
      v.rel = uint32_t(old);
    } else if (!bad && n > 0) {
      if (n > cap - len) {
        bad = true;  // longer than its row of the table: not served
      } else {
        v.need = uint32_t(((len + n + a.page - 1) >> a.page_shift) - old);
        v.want = uint32_t(n);
      }
    }
    if (bad) raise_error(AB_ERR_CAPACITY);
    return v;
  };
  auto block_scan = [&](PlanScan v, PlanScan& total) -> PlanScan {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const PlanScan y = shfl_up(v, o);
      if (lane >= o) v = v + y;
    }
    __syncthreads();  // warp_sum is reused
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    PlanScan w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const PlanScan y = shfl_up(w, o);
      if (lane >= o) w = w + y;
    }
    total = shfl_at(w, 31);
    const PlanScan before = shfl_at(w, warp - 1 < 0 ? 0 : warp - 1);
    return warp == 0 ? v : v + before;
  };

  // all pages given back (they can be handed out again in this step)
  PlanScan total{0, 0, 0}, t;
  int64_t rel_all = 0;  // at most 8 chunks of less than 2^31
  const bool one_chunk = a.S <= kPlanThreads;
  PlanScan v{0, 0, 0}, incl{0, 0, 0};
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    v = ask(s0 + tid);
    incl = block_scan(v, t);
    rel_all += t.rel;
  }
  if (F0 + rel_all > a.num_pages) {  // a page given back twice, or lists that do not belong together
    if (tid == 0) raise_error(AB_ERR_CAPACITY);
    rel_all = a.num_pages - F0;
  }
  const int F = F0 + int(rel_all);

  // the sequences up to the first that no longer fits are served
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    if (!one_chunk) {
      v = ask(s);
      incl = block_scan(v, t);
    }
    const PlanScan c = total + incl;
    if (s < a.S) {
      // sums beyond the first that does not fit are mended below
      cu_rel[s + 1] = min(int(c.rel), int(rel_all));
      cu_need[s + 1] = int(c.need) <= F && int(c.want) <= a.T ? int(c.need) : -1;
      cu_want[s + 1] = min(int(c.want), a.T);
    }
    total = total + t;
  }
  if (tid == 0) cu_want[0] = cu_need[0] = cu_rel[0] = 0;
  __syncthreads();
  if (int(total.need) > F || int(total.want) > a.T) {
    // the served sequences are a prefix: find its end, repeat its sums behind it
    if (tid == 0) raise_error(AB_ERR_CAPACITY);
    int lo = 0, hi = a.S;  // cu_need[lo] >= 0, the answer is the last such index
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (cu_need[m] >= 0) lo = m;
      else hi = m - 1;
    }
    const int need = cu_need[lo], want = cu_want[lo];
    __syncthreads();
    for (int s = lo + 1 + tid; s <= a.S; s += kPlanThreads) {
      cu_need[s] = need;
      cu_want[s] = want;
    }
    __syncthreads();
  }
  const int n_rel = cu_rel[a.S], n_need = cu_need[a.S], n_want = cu_want[a.S];

  // the last sequence whose prefix sum is <= i
  auto find = [&](const int32_t* cu, int i) -> int {
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (cu[m] <= i) lo = m;
      else hi = m - 1;
    }
    return lo;
  };
  auto given_back = [&](int i) -> int {
    const int s = find(cu_rel, i);
    return a.table[int64_t(s) * a.max_pages + (i - cu_rel[s])];
  };
  // the i-th page handed out: from the top of the list, the pages given back in this step first
  auto handed_out = [&](int i) -> int {
    const int at = F - 1 - i;
    return at >= F0 ? given_back(at - F0) : a.free_pages[at];
  };
  const int64_t gtid = int64_t(blockIdx.x) * kPlanThreads + tid, gstep = int64_t(kPlanCtas) * kPlanThreads;
  // The table rows written below (served sequences, entries from their old
  // number of pages on) are read nowhere, the list entries written (from F0 on)
  // neither.  What a thread reads first for each list is under way before it
  // writes anything.
  struct Entry {
    int64_t at;
    int page;
  };
  auto new_entry = [&](int64_t i) -> Entry {
    const int s = find(cu_need, int(i));
    const int old = (old_len[s] + a.page - 1) >> a.page_shift;
    return {int64_t(s) * a.max_pages + old + (int(i) - cu_need[s]), handed_out(int(i))};
  };
  Entry entry0{0, 0};
  int back0 = 0;
  if (gtid < n_need) entry0 = new_entry(gtid);
  if (gtid < n_rel) back0 = given_back(int(gtid));
  constexpr int kBatch = 4;  // tokens a thread looks up at once
  for (int64_t t0 = gtid; t0 < a.T; t0 += kBatch * gstep) {
    int pos[kBatch], id[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t tk = t0 + k * gstep;
      pos[k] = 0;
      id[k] = -1;
      if (tk < n_want) {
        const int s = find(cu_want, int(tk));
        const int len = old_len[s], old = (len + a.page - 1) >> a.page_shift;
        pos[k] = len + int(tk) - cu_want[s];
        const int j = pos[k] >> a.page_shift;
        id[k] = j < old ? a.table[int64_t(s) * a.max_pages + j] : handed_out(cu_need[s] + j - old);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t tk = t0 + k * gstep;
      if (tk >= a.T) break;
      int slot = -1;
      if (id[k] >= 0 && id[k] < a.num_pages) slot = (id[k] << a.page_shift) + (pos[k] & (a.page - 1));
      else if (tk < n_want) raise_error(AB_ERR_CAPACITY);
      a.slots[tk] = slot;
      a.positions[tk] = pos[k];
    }
  }
  for (int64_t i = gtid; i < n_need; i += gstep) {
    const Entry e = i == gtid ? entry0 : new_entry(i);
    a.table[e.at] = e.page;
  }
  for (int64_t i = gtid; i < n_rel; i += gstep) {
    const int page = i == gtid ? back0 : given_back(int(i));
    if (uint32_t(page) >= uint32_t(a.num_pages)) raise_error(AB_ERR_CAPACITY);  // no token can be put there either
    a.free_pages[F0 + i] = page;
  }

  // every CTA has read lens and free_count
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  for (int64_t s = gtid; s <= a.S; s += gstep) {
    a.cu_new[s] = cu_want[s];
    if (s < a.S) {
      const int len = a.lens[s];
      const bool ended = a.n_new[s] == -1 && len == old_len[s];  // a length out of range stays as it is
      a.lens_out[s] = ended ? 0 : len + cu_want[s + 1] - cu_want[s];
    }
  }
  if (gtid == 0) *a.free_count_out = F - n_need;
}

// -------------------------------------------------------------- summaries
// Mean of a page's keys, for every page that a slot list touches: the last
// written slot of each run of slots in one page owns the page, and the mean is
// over the page's keys up to that slot, without those that the call left unwritten
// (a position out of range).  A warp takes one (page, head), a run of at most 16 KB,
// eight heads a CTA.  Bound by memory (the page's keys are read once) or, for
// single tokens, by latency: 2.4 us for one token of 40 heads, about 25 us for 44
// thousand tokens of 8 heads (90 MB).

// A load that stays in its place: eight of them are under way at once.
__device__ __forceinline__ uint4 load_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

template <int D>
__global__ void __launch_bounds__(256, 4)
    page_sum_kernel(const int32_t* slots, const int32_t* positions, int n_pos, int T, int per_cta, const __nv_bfloat16* K,
                    __nv_bfloat16* ksum, int Hkv, int page_shift, int num_pages) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = blockIdx.y * 8 + warp;
  const int t0 = blockIdx.x * per_cta;
  pdl_wait();
  pdl_trigger();
  if (head >= Hkv) return;
  // positions null: no token has one
  auto refused = [&](int t) { return positions && uint32_t(__ldg(positions + t)) >= uint32_t(n_pos); };
  int slot = -1;
  if (lane < per_cta && t0 + lane < T) {
    slot = __ldg(slots + t0 + lane);
    const bool bad = refused(t0 + lane);
    if (bad || slot >> page_shift >= num_pages) slot = -1;  // reported where the token is written
    for (int t = t0 + lane + 1; slot >= 0 && t < T && __ldg(slots + t) >> page_shift == slot >> page_shift; ++t)
      if (!refused(t)) slot = -1;  // a later token is in the page
  }
  uint32_t owners = __ballot_sync(0xffffffffu, slot >= 0);
  const int sub = lane % kLanes, row0 = lane / kLanes;
  for (; owners; owners &= owners - 1) {
    const int owner = t0 + __ffs(owners) - 1, sl = __shfl_sync(0xffffffffu, slot, owner - t0);
    const int64_t id = sl >> page_shift;
    const int n = (sl & ((1 << page_shift) - 1)) + 1;
    // the up to 63 tokens before it in the list, for those of its page that were refused
    int before[2] = {-1, -1}, at[2] = {0, 0};
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int t = owner - 1 - lane - 32 * z;
      if (positions && t >= 0 && 32 * z < n - 1) {
        before[z] = __ldg(slots + t);
        at[z] = __ldg(positions + t);
      }
    }
    uint64_t holes = 0;  // of the page's keys
    const __nv_bfloat16* src = K + (((id * Hkv + head) << page_shift) * D) + sub * 8;
    float acc[8] = {};
    for (int r0 = 0; r0 < n; r0 += 8 * kRows) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + k * kRows + row0;
        x[k] = r < n ? load_16(src + int64_t(r) * D) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (r0 == 0) {
        uint64_t mine = 0;
#pragma unroll
        for (int z = 0; z < 2; ++z)
          if (before[z] < sl && before[z] >> page_shift == sl >> page_shift && uint32_t(at[z]) >= uint32_t(n_pos))
            mine |= uint64_t(1) << (before[z] & ((1 << page_shift) - 1));
        holes = uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(mine))) |
                uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(mine >> 32))) << 32;
      }
      if (holes) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + k * kRows + row0;
          if (r < n && (holes >> r) & 1) x[k] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * e] += __uint_as_float(u[e] << 16);
          acc[2 * e + 1] += __uint_as_float(u[e] & 0xFFFF0000u);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      acc[e] /= float(n - __popcll(holes));
    }
    if (row0 == 0)
      *reinterpret_cast<uint4*>(ksum + (id * Hkv + head) * D + sub * 8) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                     pack_bf16x2(acc[6], acc[7]));
  }
}

// ------------------------------------------------- an even share of ragged work
// The work is a list of units, each of `rows` rows of `tiles` equal tiles.  A
// row costs two for each tile and `row_cost` besides; CTA c of C takes the tiles
// between c / C and (c + 1) / C of the whole cost, whatever the units' lengths,
// so the load is even without the host knowing any length.  Every CTA sums the
// units itself.  With `whole` a row belongs to the CTA in whose share it begins.
struct UnitWork {
  int rows, tiles;  // tiles of each row
};
struct Share {
  int unit;   // first unit with work
  int off;    // first tile in it (may be one past its last: the next unit then)
  int n;      // tiles of this CTA
  int begin;  // position of the first tile in the whole list
};

__device__ __forceinline__ int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

constexpr int kShareMaxUnits = 65536;
constexpr int kShareSums = kShareMaxUnits / 32;  // pairs of sums over 32 units each

// Sums stay below 2^31: the host limits the tiles of a full table to 2^29.
template <typename F>
__device__ __forceinline__ Share share_work(F work, int row_cost, bool whole, int n_units, int c, int C, int2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int chunks = (n_units + 31) / 32;
  auto unit_work = [&](int u) { return u < n_units ? work(u) : UnitWork{0, 0}; };
  auto cost_of = [&](const UnitWork& w) { return w.tiles > 0 ? w.rows * (2 * w.tiles + row_cost) : 0; };
  // the two ends of the share: cost p, and its chunk of 32 units with the sums before it
  int p[2], chunk[2] = {0, 0}, base[2] = {0, 0}, before[2] = {0, 0}, total_tiles;
  UnitWork w[2];
  auto ends = [&](int total) {
    const int q = total / C, r = total - q * C;
    p[0] = c * q + min(c, r);
    p[1] = p[0] + q + (c < r ? 1 : 0);
  };
  int total;
  if (chunks == 1) {
    w[0] = w[1] = unit_work(lane);
    total = __reduce_add_sync(0xffffffffu, cost_of(w[0]));
    total_tiles = __reduce_add_sync(0xffffffffu, w[0].rows * w[0].tiles);
    ends(total);
  } else {
    for (int k = warp; k < chunks; k += warps) {
      const UnitWork x = unit_work(k * 32 + lane);
      const int cost = __reduce_add_sync(0xffffffffu, cost_of(x));
      const int tiles = __reduce_add_sync(0xffffffffu, x.rows * x.tiles);
      if (lane == 0) sums[k] = make_int2(cost, tiles);
    }
    __syncthreads();
    // every warp works its CTA's share out by itself
    total = total_tiles = 0;
    for (int k = lane; k < chunks; k += 32) {
      total += sums[k].x;
      total_tiles += sums[k].y;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    total_tiles = __reduce_add_sync(0xffffffffu, total_tiles);
    ends(total);
    int cost = 0, tiles = 0;  // of the chunks before
    bool open[2] = {true, true};
    for (int k0 = 0; k0 < chunks && (open[0] || open[1]); k0 += 32) {
      const int2 x = k0 + lane < chunks ? sums[k0 + lane] : make_int2(0, 0);
      const int incl = warp_inclusive(x.x), incl_tiles = warp_inclusive(x.y);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t past = __ballot_sync(0xffffffffu, cost + incl > p[z]);
        if (open[z] && past) {
          const int l = __ffs(past) - 1;
          chunk[z] = k0 + l;
          base[z] = cost + __shfl_sync(0xffffffffu, incl - x.x, l);
          before[z] = tiles + __shfl_sync(0xffffffffu, incl_tiles - x.y, l);
          open[z] = false;
        }
      }
      cost += __shfl_sync(0xffffffffu, incl, 31);
      tiles += __shfl_sync(0xffffffffu, incl_tiles, 31);
    }
    w[0] = unit_work(chunk[0] * 32 + lane);
    w[1] = unit_work(chunk[1] * 32 + lane);
  }
  // the first tile at or behind cost p: its unit, place in the unit, place in the list
  int unit[2], off[2], at[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const int cost = cost_of(w[z]), incl = warp_inclusive(cost), tiles = w[z].rows * w[z].tiles;
    const int incl_tiles = warp_inclusive(tiles);
    const int l = __ffs(__ballot_sync(0xffffffffu, base[z] + incl > p[z]) | 0x80000000u) - 1;
    const int rest = p[z] - base[z] - __shfl_sync(0xffffffffu, incl - cost, l);
    const int T = __shfl_sync(0xffffffffu, w[z].tiles, l), row_total = 2 * T + row_cost;
    const int row = row_total > 0 ? rest / row_total : 0, x = rest - row * row_total;
    unit[z] = chunk[z] * 32 + l;
    off[z] = row * T + (whole ? (x > 0 ? T : 0) : min((x + 1) / 2, T));
    at[z] = before[z] + __shfl_sync(0xffffffffu, incl_tiles - tiles, l) + off[z];
    if (p[z] >= total) {
      unit[z] = n_units;
      off[z] = 0;
      at[z] = total_tiles;
    }
  }
  return Share{unit[0], off[0], at[1] - at[0], at[0]};
}

// First unit from u on with tiles, n_units if there is none; whole warps, 32
// units at a time.
template <typename F>
__device__ __forceinline__ int next_unit(F tiles, int n_units, int u) {
  const int lane = threadIdx.x & 31;
  for (; u < n_units; u += 32) {
    const uint32_t some = __ballot_sync(0xffffffffu, u + lane < n_units && tiles(u + lane) > 0);
    if (some) return u + __ffs(some) - 1;
  }
  return n_units;
}

// m16n8k16 bf16 product with fp32 accumulation.  The single-token kernels use
// it instead of tcgen05: a key meets at most 16 queries, so they are bound by
// the bytes of the keys, and operands straight from registers need neither a
// 128-row tile nor a trip through TMEM.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ----------------------------------------------------------------- select
// P[s, g, j] = (1/G) sum_h softmax_j(q_h . kbar_j / sqrt(d) + ln n_j): the
// block-mass estimate of the selector with the group's G query heads in the
// place of the clusters.  Two kernels: the scores (and each chunk's maximum
// and sum of exponentials per head) go to the workspace, then every chunk is
// normalised with the row's sums.
//
// Scores: a warp takes 32 pages of one head, four products of 8 pages.  The
// order of the d products is free, so lane (g, t) takes the 16-byte pieces t,
// t + 4, ... of page g's summary and the query's registers follow the same
// order: what a lane needs it copies itself, one step of 32 pages ahead of its
// use (cp.async into its own places, no barrier).  Bound by memory: 2 d bytes
// of summary per page and head, and 8 G for its scores, mostly in L2.  48
// sequences of 62 thousand tokens, 8 key heads of 4: 73 us for 401 MB (5.5 TB/s),
// and 8 us for the normalisation.
constexpr int kSelPages = 32;
constexpr int kSelWarps = 8;  // 9 to 14: the same time, with 32 key heads 437 us against 266
__host__ __device__ constexpr int sel_stages(int D) { return D == 128 ? 3 : 6; }

struct SelectArgs {
  PagedView v;
  const __nv_bfloat16* Q;     // [T, Hq, d]
  const __nv_bfloat16* ksum;  // [num_pages, Hkv, d]
  float* scores;              // [S, Hkv, G, pitch], log2 domain
  float2* part;               // [S, Hkv, G, chunks]: maximum, sum of exp2
  float* P;                   // [S, Hkv, max_pages]
  int chunks;                 // ceil(max_pages / 32)
  int pitch;                  // max_pages rounded up to a multiple of 4
  float scale_log2;
};

// kWide: more than 8 query heads per key/value head.
template <int D, bool kWide>
__global__ void __launch_bounds__(kSelWarps * 32, 1) page_score_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kPieces = D / 32;  // 16-byte pieces of a summary per lane
  constexpr int kStages = sel_stages(D);
  constexpr int kHalves = kWide ? 2 : 1;  // blocks of 8 heads
  extern __shared__ uint4 sel_smem[];  // [warps][stages][4 kPieces][32 lanes]
  __shared__ int2 sums[kMaxSeqs / 32];
  pdl_wait();
  pdl_trigger();
  const PagedView& v = a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  auto chunks_of = [&](int s) {
    return query_row(v, s) < 0 ? 0 : (pages_of(v, seq_len(v, s)) + kSelPages - 1) / kSelPages;
  };
  auto work = [&](int s) { return UnitWork{v.Hkv, chunks_of(s)}; };
  const Share sh = share_work(work, 0, false, v.S, blockIdx.x, gridDim.x, sums);
  uint4* const mine = sel_smem + size_t(warp) * kStages * 4 * kPieces * 32 + lane;
  const int n_steps = (sh.n - warp + kSelWarps - 1) / kSelWarps;  // this warp's: every 8th of the CTA's
  if (n_steps <= 0) return;

  // A step is head hk of pages [32 chunk, 32 chunk + 32) of sequence s; heads
  // are innermost, so the warps of a CTA read neighbouring heads of the same
  // pages at about the same time (a page's summaries are contiguous).
  struct Step {
    int s, pages, len, row, chunk, hk;  // row: of Q
  };
  auto open_seq = [&](Step& x) {
    x.len = seq_len(v, x.s);
    x.pages = pages_of(v, x.len);
    x.row = query_row(v, x.s);
  };
  auto settle = [&](Step& x) -> bool {  // the step `hk` heads behind the start of its chunk
    while (x.hk >= v.Hkv) {
      x.hk -= v.Hkv;
      if (++x.chunk * kSelPages >= x.pages) {
        x.chunk = 0;
        x.s = next_unit([&](int s) { return chunks_of(s); }, v.S, x.s + 1);
        if (x.s >= v.S) return false;
        open_seq(x);
      }
    }
    return true;
  };
  Step cur{sh.unit, 0, 0, 0, sh.off / v.Hkv, 0};
  open_seq(cur);
  cur.hk = sh.off - cur.chunk * v.Hkv + warp;
  if (cur.chunk * kSelPages >= cur.pages) {  // one past the unit's last step
    --cur.chunk;
    cur.hk += v.Hkv;
  }
  if (!settle(cur)) return;

  // copies, kStages - 1 steps ahead
  Step ahead = cur;
  int left_ahead = n_steps;
  int id[4];  // this lane's pages of the step ahead, as read: looked at when they are copied
  auto look_up = [&]() {
    const int32_t* from = v.table + int64_t(ahead.s) * v.max_pages + ahead.chunk * kSelPages + g;
#pragma unroll
    for (int n = 0; n < 4; ++n) id[n] = ahead.chunk * kSelPages + n * 8 + g < ahead.pages ? __ldg(from + n * 8) : 0;
  };
  look_up();
  auto copy_next = [&](int stage) {
    if (left_ahead > 0) {
      uint4* dst = mine + stage * 4 * kPieces * 32;
      const __nv_bfloat16* base = a.ksum + int64_t(ahead.hk) * D + t * 8;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const bool there = uint32_t(id[n]) < uint32_t(v.num_pages);
        if (!there) raise_error(AB_ERR_CAPACITY);  // its score is that of a zero summary
        const __nv_bfloat16* src = base + int64_t(id[n]) * v.Hkv * D;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          if (there) cp_async16(smem_u32(dst + (n * kPieces + p) * 32), src + p * 32);
          else dst[(n * kPieces + p) * 32] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (--left_ahead > 0) {
        const int s = ahead.s, chunk = ahead.chunk;
        ahead.hk += kSelWarps;
        if (!settle(ahead)) left_ahead = 0;
        else if (ahead.s != s || ahead.chunk != chunk) look_up();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) copy_next(k);

  // query: rows g (and g + 8) of the 16 x d operand, pieces in the keys' order,
  // read a step ahead
  uint4 qx[kHalves][kPieces], qn[kHalves][kPieces];
  auto read_query = [&](const Step& x) {
    const __nv_bfloat16* q = a.Q + ((int64_t(x.row) * v.Hkv + x.hk) * v.G + g) * D + t * 8;
#pragma unroll
    for (int k = 0; k < kHalves; ++k)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        qn[k][p] = g + 8 * k < v.G ? __ldg(reinterpret_cast<const uint4*>(q + k * 8 * D + p * 32)) : make_uint4(0u, 0u, 0u, 0u);
  };
  read_query(cur);
  int stage = 0;
  for (int left = n_steps; left > 0; --left) {
    copy_next(stage == 0 ? kStages - 1 : stage - 1);
#pragma unroll
    for (int k = 0; k < kHalves; ++k)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) qx[k][p] = qn[k][p];
    Step nxt = cur;
    if (left > 1) {
      nxt.hk += kSelWarps;
      if (settle(nxt)) read_query(nxt);
      else left = 1;
    }
    const int64_t row = (int64_t(cur.s) * v.Hkv + cur.hk) * v.G + g;
    cp_async_wait<kStages - 1>();
    const uint4* kx = mine + stage * 4 * kPieces * 32;
    float x[kHalves][8];
    const float bias = float(v.page_shift);  // log2 of a whole page's keys
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float c0[4] = {}, c1[4] = {};
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint4 k = kx[(n * kPieces + p) * 32];
        const uint4 q0 = qx[0][p], q1 = kWide ? qx[kHalves - 1][p] : make_uint4(0u, 0u, 0u, 0u);
        mma_16816(c0, q0.x, q1.x, q0.y, q1.y, k.x, k.y);
        mma_16816(c1, q0.z, q1.z, q0.w, q1.w, k.z, k.w);
      }
#pragma unroll
      for (int k = 0; k < kHalves; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) x[k][2 * n + e] = fmaf(c0[2 * k + e] + c1[2 * k + e], a.scale_log2, bias);
    }
    const int rest = cur.pages - cur.chunk * kSelPages;  // pages of this chunk and behind
    if (rest <= kSelPages) {  // the last page may have fewer keys, behind it there is none
      const float last_bias = log2f(float(cur.len - ((cur.pages - 1) << v.page_shift))) - bias;
#pragma unroll
      for (int k = 0; k < kHalves; ++k)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int j = (n >> 1) * 8 + t * 2 + (n & 1);
          if (j == rest - 1) x[k][n] += last_bias;
          if (j >= rest) x[k][n] = -INFINITY;
        }
    }
#pragma unroll
    for (int k = 0; k < kHalves; ++k) {
      float m = -INFINITY;
#pragma unroll
      for (int n = 0; n < 8; ++n) m = fmaxf(m, x[k][n]);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int n = 0; n < 8; ++n) l += ex2_approx(x[k][n] - ref);
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (g + 8 * k < v.G) {
        if (t == 0) a.part[(row + 8 * k) * a.chunks + cur.chunk] = make_float2(m, l);
        float* dst = a.scores + (row + 8 * k) * a.pitch + cur.chunk * kSelPages + t * 2;
        if (rest >= kSelPages) {
#pragma unroll
          for (int n = 0; n < 4; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(x[k][2 * n], x[k][2 * n + 1]);
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n)  // up to the end of a group of 4: the pitch is a multiple of it
            if (n * 8 + t * 2 < ((rest + 3) & ~3))
              *reinterpret_cast<float2*>(dst + n * 8) = make_float2(x[k][2 * n], x[k][2 * n + 1]);
        }
      }
    }
    cur = nxt;
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// Normalisation: every CTA joins the row's partial sums, then turns 1024
// pages' scores into P, at most 8 steps apart along the row.
constexpr int kNormThreads = 256;

__global__ void __launch_bounds__(kNormThreads) page_mass_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ float2 ml[kMaxGroup];  // maximum, 1 / (G sum)
  pdl_wait();
  pdl_trigger();
  const PagedView& v = a.v;
  const int s = blockIdx.z, hk = blockIdx.y;
  if (query_row(v, s) < 0) return;
  const int pages = pages_of(v, seq_len(v, s));
  if (int(blockIdx.x) * 4 * kNormThreads >= pages) return;
  const int chunks = (pages + kSelPages - 1) / kSelPages;
  const int64_t row = int64_t(s) * v.Hkv + hk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int h = warp; h < v.G; h += kNormThreads / 32) {
    const float2* part = a.part + (row * v.G + h) * a.chunks;
    float m = -INFINITY, l = 0.f;
    for (int k0 = lane; k0 < chunks; k0 += 128) {
      float2 z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = k0 + 32 * k < chunks ? part[k0 + 32 * k] : make_float2(-INFINITY, 0.f);
      const float mm = fmaxf(fmaxf(fmaxf(z[0].x, z[1].x), fmaxf(z[2].x, z[3].x)), m);
      const float ref = mm == -INFINITY ? 0.f : mm;
      l *= exp2f(m - ref);
#pragma unroll
      for (int k = 0; k < 4; ++k) l += z[k].y * exp2f(z[k].x - ref);
      m = mm;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o);
      const float mm = fmaxf(m, om), ref = mm == -INFINITY ? 0.f : mm;
      l = l * exp2f(m - ref) + ol * exp2f(om - ref);
      m = mm;
    }
    if (lane == 0) ml[h] = make_float2(m, 1.f / (l * float(v.G)));
  }
  __syncthreads();
  for (int j = (blockIdx.x * kNormThreads + threadIdx.x) * 4; j < pages; j += gridDim.x * 4 * kNormThreads) {
    const float* src = a.scores + row * v.G * a.pitch + j;
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int h = 0; h < v.G; ++h) {
      const float4 x = *reinterpret_cast<const float4*>(src + int64_t(h) * a.pitch);
      const float2 z = ml[h];
      p.x += ex2_approx(x.x - z.x) * z.y;
      p.y += ex2_approx(x.y - z.x) * z.y;
      p.z += ex2_approx(x.z - z.x) * z.y;
      p.w += ex2_approx(x.w - z.x) * z.y;
    }
    float* dst = a.P + row * v.max_pages + j;
    dst[0] = p.x;
    if (j + 1 < pages) dst[1] = p.y;
    if (j + 2 < pages) dst[2] = p.z;
    if (j + 3 < pages) dst[3] = p.w;
  }
}

// The whole selection of a row in one launch, for tables of few pages: a CTA
// takes a (sequence, key/value head), eight warps 32 pages at a time, and the
// scores stay in shared memory.  Bound by latency (table, then summaries, then
// the join of the warps): 2.6 us for 3 sequences of 12 heads and 47 pages, 3.5
// for 8 of 8 heads and 256.
constexpr int kRowPages = 1024;                      // columns of the table at most
constexpr int64_t kRowBytes = int64_t(160) << 20;    // of all summaries of a full table
constexpr int kRowThreads = 256;

template <int D, bool kWide>
__global__ void __launch_bounds__(kRowThreads) page_row_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kPieces = D / 32;
  constexpr int kHalves = kWide ? 2 : 1;
  constexpr int kWarps = kRowThreads / 32;
  extern __shared__ float row_smem[];  // [G][pitch] scores, log2 domain
  __shared__ float2 wpart[kWarps][kMaxGroup];
  pdl_wait();
  pdl_trigger();
  const PagedView& v = a.v;
  const int s = blockIdx.x / v.Hkv, hk = blockIdx.x - s * v.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int qrow = query_row(v, s);
  if (qrow < 0) return;
  const int len = seq_len(v, s), pages = pages_of(v, len);
  // queries: rows g (and g + 8) of the 16 x d operand, 16-byte pieces t, t + 4, ...
  const __nv_bfloat16* q = a.Q + ((int64_t(qrow) * v.Hkv + hk) * v.G + g) * D + t * 8;
  uint4 qx[kHalves][kPieces];
#pragma unroll
  for (int k = 0; k < kHalves; ++k)
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      qx[k][p] = g + 8 * k < v.G ? __ldg(reinterpret_cast<const uint4*>(q + k * 8 * D + p * 32)) : make_uint4(0u, 0u, 0u, 0u);
  float m[kHalves], l[kHalves];
#pragma unroll
  for (int k = 0; k < kHalves; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
  }
  const float bias = float(v.page_shift);  // log2 of a whole page's keys
  const float last_bias = log2f(float(len - ((pages - 1) << v.page_shift)));
  for (int j0 = warp * 32; j0 < pages; j0 += kWarps * 32) {
    int id[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      id[n] = j0 + n * 8 + g < pages ? __ldg(v.table + int64_t(s) * v.max_pages + j0 + n * 8 + g) : 0;
    uint4 kx[4][kPieces];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const bool there = uint32_t(id[n]) < uint32_t(v.num_pages);
      if (!there) raise_error(AB_ERR_CAPACITY);  // its score is that of a zero summary
      const __nv_bfloat16* src = a.ksum + (int64_t(id[n]) * v.Hkv + hk) * D + t * 8;
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        kx[n][p] = there ? __ldg(reinterpret_cast<const uint4*>(src + p * 32)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float x[kHalves][8];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float c0[4] = {}, c1[4] = {};
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint4 q0 = qx[0][p], q1 = kWide ? qx[kHalves - 1][p] : make_uint4(0u, 0u, 0u, 0u), k = kx[n][p];
        mma_16816(c0, q0.x, q1.x, q0.y, q1.y, k.x, k.y);
        mma_16816(c1, q0.z, q1.z, q0.w, q1.w, k.z, k.w);
      }
#pragma unroll
      for (int k = 0; k < kHalves; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = j0 + n * 8 + t * 2 + e;
          x[k][2 * n + e] = j >= pages ? -INFINITY
                                       : fmaf(c0[2 * k + e] + c1[2 * k + e], a.scale_log2, j == pages - 1 ? last_bias : bias);
        }
    }
#pragma unroll
    for (int k = 0; k < kHalves; ++k) {
      float mx = m[k];
#pragma unroll
      for (int n = 0; n < 8; ++n) mx = fmaxf(mx, x[k][n]);
      // this lane's maximum and sum; a quad's are joined at the end
      const float ref = mx == -INFINITY ? 0.f : mx;
      l[k] *= ex2_approx(m[k] - ref);
#pragma unroll
      for (int n = 0; n < 8; ++n) l[k] += ex2_approx(x[k][n] - ref);
      m[k] = mx;
      if (g + 8 * k < v.G) {
        float* dst = row_smem + (g + 8 * k) * a.pitch + j0 + t * 2;
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (j0 + n * 8 + t * 2 < a.pitch) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(x[k][2 * n], x[k][2 * n + 1]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kHalves; ++k) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m[k], o), ol = __shfl_xor_sync(0xffffffffu, l[k], o);
      const float mm = fmaxf(m[k], om), ref = mm == -INFINITY ? 0.f : mm;
      l[k] = l[k] * ex2_approx(m[k] - ref) + ol * ex2_approx(om - ref);
      m[k] = mm;
    }
    if (t == 0) wpart[warp][g + 8 * k] = make_float2(m[k], l[k]);
  }
  __syncthreads();
  if (threadIdx.x < v.G) {  // the head's maximum, and 1 / (G sum)
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, wpart[w][threadIdx.x].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 z = wpart[w][threadIdx.x];
      ll += z.y * exp2f(z.x - (mm == -INFINITY ? 0.f : mm));
    }
    wpart[0][threadIdx.x] = make_float2(mm, 1.f / (ll * float(v.G)));
  }
  __syncthreads();
  float* P = a.P + int64_t(blockIdx.x) * v.max_pages;
  for (int j = threadIdx.x; j < pages; j += kRowThreads) {
    float p = 0.f;
    for (int h = 0; h < v.G; ++h) p += ex2_approx(row_smem[h * a.pitch + j] - wpart[0][h].x) * wpart[0][h].y;
    P[j] = p;
  }
}

// ------------------------------------------------------------------- top-k
// The newest min(recent, Kb) pages and the Kb minus that many others of
// largest P, in ascending order; ties go to the lower page.  Keys are P's bits
// (P >= 0 orders as its bits; anything else counts as 0), the newest pages get
// the largest key.  One CTA per row, the row's keys in shared memory: a radix
// select over digits of 11, 11 and 9 bits (the first holds exponent and three
// bits of the fraction, so that the counters of a row's few octaves do not
// collide), then every thread writes the kept pages of its own run of the row.
// Where at most 256 keys share the first digit of the last one kept, they are
// gathered and counted in place of the other digits (320 rows of 2047 pages: 8.2
// us, 9.7 by digits).
// Rows of at most 256 pages count instead how many keys come before each.
// (2048 rows of 128 pages: 8.9 us, 20.2 by digits; 10 rows of 79: 2.0 and 4.0).
// Bound by the latency of the steps: 256 threads for tables of up to 2560 pages
// (2047 pages in 320 rows by digits: 9.7 us, with 512 threads 10.8), 512 up to 8192 (4096
// pages in 512 rows: 14.8 us, 17.8 with 256), else 1024 (one row of 20000 pages:
// 13.9 us, 18.4 with 512).
struct TopkArgs {
  const float* P;
  const int32_t* lens;
  int32_t *idx, *count;
  int Hkv, page, page_shift, max_pages, recent;
  int cap;  // keys that fit in shared memory (longer rows are read anew in each step)
  double keep;
};
constexpr int kTopkCount = 256;      // pages of a row that is counted
constexpr int kTopkMaxKeys = 24576;  // 96 KB: two CTAs an SM
constexpr int kTopkBins = 2048;

__device__ __forceinline__ int page_budget(int n, double keep) {
  const double kb = floor(keep * double(n) + 0.5);
  return kb < 1.0 ? min(1, n) : kb > double(n) ? n : int(kb);
}

template <int kTopkThreads>
__global__ void __launch_bounds__(kTopkThreads) page_topk_kernel(const __grid_constant__ TopkArgs a) {
  extern __shared__ uint4 topk_smem[];
  uint32_t* const topk_keys = reinterpret_cast<uint32_t*>(topk_smem);
  __shared__ uint32_t hist[kTopkBins];
  __shared__ uint32_t sel[4];  // digit (key), how many of its keys are kept, how many there are; keys gathered
  __shared__ uint32_t wsum[2][kTopkThreads / 32];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  int len = __ldg(a.lens + row / a.Hkv);
  if (len < 0 || len > a.max_pages << a.page_shift) {
    if (tid == 0) raise_error(AB_ERR_CAPACITY);
    len = 0;
  }
  const int n = (len + a.page - 1) >> a.page_shift;
  const int Kb = page_budget(n, a.keep);
  if (tid == 0) a.count[row] = Kb;
  if (n == 0) return;
  const int newest = n - min(a.recent, Kb);  // pages from here on are kept
  const float* P = a.P + int64_t(row) * a.max_pages;
  auto make_key = [&](int j, float p) -> uint32_t {
    return j >= newest ? 0x7FFFFFFFu : p > 0.f ? __float_as_uint(p) : 0u;
  };
  int32_t* out = a.idx + int64_t(row) * a.max_pages;
  if (n <= kTopkCount) {
    static_assert(kTopkCount <= kTopkThreads, "a thread per page");
    const int j = tid;
    const uint32_t mine = j < n ? make_key(j, __ldg(P + j)) : 0u;
    if (j < kTopkCount) topk_keys[j] = mine;  // 0 behind the row: it comes before nothing
    __syncthreads();
    // keys before this one: larger, or equal and of a lower page
    int rank = 0;
    if (warp * 32 < n) {
      const int below = j >> 2;  // groups of four pages below this one's group
      for (int i = 0; i < (n + 3) >> 2; ++i) {
        const uint4 k = topk_smem[i];
        const uint32_t least = mine + (i < below ? 0u : 1u);
        rank += int(k.x >= least) + int(k.y >= least) + int(k.z >= least) + int(k.w >= least);
      }
      for (int i = j & ~3; i < j; ++i) rank += int(topk_keys[i] == mine);
    }
    const bool kept = j < n && rank < Kb;
    const uint32_t some = __ballot_sync(0xffffffffu, kept);
    if (lane == 0) wsum[0][warp] = uint32_t(__popc(some));
    __syncthreads();
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[0][lane] : 0u);
    if (kept) out[before + __popc(some & ((1u << lane) - 1u))] = j;
    return;
  }
  const bool cached = n <= a.cap;
  if (tid == 0) sel[3] = 0;
  if (cached) {
    for (int j0 = tid; j0 < n; j0 += 4 * kTopkThreads) {
      float p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = j0 + k * kTopkThreads < n ? __ldg(P + j0 + k * kTopkThreads) : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j0 + k * kTopkThreads < n) topk_keys[j0 + k * kTopkThreads] = make_key(j0 + k * kTopkThreads, p[k]);
    }
  }
  auto key_of = [&](int j) -> uint32_t { return cached ? topk_keys[j] : make_key(j, __ldg(P + j)); };
  // inclusive sums over the block's threads of two counts
  auto block_scan = [&](uint32_t& x, uint32_t& y) {
    const uint32_t x0 = x, y0 = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += p;
        y += q;
      }
    }
    if (lane == 31) {
      wsum[0][warp] = x;
      wsum[1][warp] = y;
    }
    __syncthreads();
    uint32_t p = lane < warp ? wsum[0][lane] : 0u, q = lane < warp ? wsum[1][lane] : 0u;
    p = __reduce_add_sync(0xffffffffu, p);
    q = __reduce_add_sync(0xffffffffu, q);
    x += p - x0;  // exclusive
    y += q - y0;
  };
  uint32_t prefix = 0, pmask = 0, need = uint32_t(Kb);
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 20 : pass == 1 ? 9 : 0;
    const uint32_t digits = pass == 2 ? 511u : 2047u;
    for (int k = tid; k < kTopkBins; k += kTopkThreads) hist[k] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kTopkThreads) {
      const uint32_t k = key_of(j);
      if ((k & pmask) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1u);
    }
    __syncthreads();
    // thread t: bins 2047 - 4 t down to 2044 - 4 t
    constexpr int kPer = kTopkBins / kTopkThreads;
    uint32_t c[kPer], tot = 0, none = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      c[k] = hist[kTopkBins - 1 - kPer * tid - k];
      tot += c[k];
    }
    uint32_t above = tot;
    block_scan(above, none);
    if (above < need && need <= above + tot) {  // exactly one thread
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (above < need && need <= above + c[k]) {
          sel[0] = uint32_t(kTopkBins - 1 - kPer * tid - k);
          sel[1] = need - above;
          sel[2] = c[k];
        }
        above += c[k];
      }
    }
    __syncthreads();
    prefix |= sel[0] << shift;
    pmask |= digits << shift;
    need = sel[1];
    const uint32_t rest = sel[2];
    if (pass == 0 && rest <= kTopkCount) {
      // few keys share the digit: gather them (in hist) and count instead
      for (int j0 = warp * 32; j0 < n; j0 += kTopkThreads) {
        const int j = j0 + lane;
        const uint32_t k = j < n ? key_of(j) : 0u;
        const bool among = j < n && (k & pmask) == prefix;
        const uint32_t some = __ballot_sync(0xffffffffu, among);
        if (some == 0) continue;
        uint32_t at = 0;
        if (lane == 0) at = atomicAdd(&sel[3], uint32_t(__popc(some)));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(some & ((1u << lane) - 1u));
        if (among) {
          hist[at] = k;
          hist[kTopkCount + at] = uint32_t(j);
        }
      }
      __syncthreads();
      if (tid < int(rest)) {
        const uint32_t k = hist[tid], j = hist[kTopkCount + tid];
        uint32_t larger = 0, equal = 0;  // equal: of a lower page
        for (uint32_t i = 0; i < rest; ++i) {
          larger += hist[i] > k ? 1u : 0u;
          equal += hist[i] == k && hist[kTopkCount + i] < j ? 1u : 0u;
        }
        if (larger + equal == need - 1) {  // exactly one: the last that is kept
          sel[0] = k;
          sel[1] = equal + 1;
        }
      }
      __syncthreads();
      prefix = sel[0];
      need = sel[1];
      break;
    }
  }
  // kept: keys above the threshold, and the lowest `need` pages of those equal to it
  const int per = (n + kTopkThreads - 1) / kTopkThreads, first = tid * per, last = min(first + per, n);
  uint32_t n_gt = 0, n_eq = 0;
  for (int j = first; j < last; ++j) {
    const uint32_t k = key_of(j);
    n_gt += k > prefix ? 1u : 0u;
    n_eq += k == prefix ? 1u : 0u;
  }
  block_scan(n_gt, n_eq);
  for (int j = first; j < last; ++j) {
    const uint32_t k = key_of(j);
    const bool gt = k > prefix, eq = k == prefix;
    if (gt || (eq && n_eq < need)) out[n_gt + min(n_eq, need)] = j;
    n_gt += gt ? 1u : 0u;
    n_eq += eq ? 1u : 0u;
  }
}

}  // namespace ab
