// Norms of queries and keys with the position rotation, in one pass from the
// projections' layout (tokens outermost, any strides) to the attention's:
// [B, H, L, d], or the new tokens' Q and the pages of a key-value cache.
//
// For a head's values x of one token, all in fp32 with one rounding to
// bfloat16 at the end:
//   y_i = x_i r w_i,  r = 1/sqrt(mean(x^2) + eps) over the head (norm 1) or
//                     over all heads of the token (norm 2); r = 1 for norm 0
//   (a, b) -> (a cos - b sin, a sin + b cos) for the pairs (2i, 2i+1)
//                     (interleaved) or (i, i + d/2); table row = position
//
// Bound by memory, with the instructions close behind (2 bytes in and 2 bytes
// out per value).  A head's d values lie in d / 8 lanes of 16 bytes, so every
// access is a whole head row (128 or 256 bytes).  A lane copies its own pieces
// into shared memory (cp.async) some steps ahead, the token's table row with
// them, and registers hold only the weights and the row's cos and sin.  For the
// pairs (i, i + d/2) a lane reads back four values of each half, which spares
// eight shuffles a row.
//  - norm 0 and 1: a warp takes a unit of one token and some or all of its heads
//    (all where there are tokens enough: the unit's addresses and table row are
//    then worked out once), four head rows a lane in a step.  The units of q, k
//    and v go token by token, so that a fused projection is read front to back.
//  - norm 2: a CTA takes a token of one tensor at a time, tensor after tensor,
//    so that the weights of its lanes' heads stay in registers; r goes into cos
//    and sin.
// Measured on 32760 tokens of 40 heads of 128, q, k and v (2.03 GB): norm 2
// 351 us (5.8 TB/s), norm 1 355, rotation alone 346; with one CTA a token and
// nothing copied ahead norm 2 took 473.  Copies of rows to places a sequence apart
// keep the last tenth of the copy rate away: rotation alone is no faster.
#pragma once

#include "ab_ptx.cuh"

namespace ab {

enum : int { kNormNone = 0, kNormHead = 1, kNormToken = 2 };

// A token tensor: value i of head h of token t of batch element b lies at
// ptr + b * sb + t * st + h * sh + i (elements).
struct TokenView {
  const __nv_bfloat16* ptr;
  int64_t sb, st, sh;
};

struct NormRopeArgs {
  TokenView in[3];         // q, k, v; ptr null: this one is not wanted
  __nv_bfloat16* out[3];
  const float* w[2];       // weights of q and k, null: ones
  const int32_t* pos[3];   // positions of the tokens, null: the token's index (v's: in the paged destination only)
  const float *cos_t, *sin_t;  // [n_pos, d/2], both null: no rotation
  int n_pos;
  float eps;
  int heads[3];
  int len[3];              // tokens per batch element
  int tokens[3];           // tokens in all
  int units[3];            // end of each one's units in the list; if merged, of each one's units within a token
  int steps[3];            // steps of a unit
  bool merged;             // token by token (all three have the same tokens)
  int n_units;
  // paged destination
  const int32_t* slots;    // [T], null: the dense destination
  int page_shift, num_pages;
};

// The kernels of the paged path are launched while the kernel before them in
// the stream still runs, and wait here for its end and its results; pdl_trigger
// lets the next one be launched.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// acc += v^2 for both bf16 halves of v: products with bf16 operands, fp32 sums.
__device__ __forceinline__ void square_add(uint32_t v, float& acc) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
      "fma.rn.f32.bf16 %0, lo, lo, %0;\n\tfma.rn.f32.bf16 %0, hi, hi, %0;\n\t}"
      : "+f"(acc)
      : "r"(v));
}

constexpr int kRopeThreads = 128;  // of a CTA whose warps take units of their own
constexpr int kRopeRows = 4;       // head rows a lane takes in a step
constexpr int kRopeRowsMany = 8;   // of a CTA per token whose 16 warps would not hold its heads by fours
constexpr int kRopeStages = 4, kRopeStagesMany = 2;  // steps in flight

// Bytes of shared memory: the pieces, the table rows, and the place per warp.
__host__ __device__ constexpr int rope_smem_bytes(int nv, int stages, int threads) {
  return stages * threads * 16 * (nv + 1) + stages * (threads / 32) * 16;
}

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(x[k] << 16);
    f[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float sum_squares8(const uint4& v) {
  float q0 = 0.f, q1 = 0.f;
  square_add(v.x, q0);
  square_add(v.y, q1);
  square_add(v.z, q0);
  square_add(v.w, q1);
  return q0 + q1;
}
__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Which 8 values of a head row lane `sub` of the row's kLanes takes: 8 in a row
// where the pairs are neighbours, else four of each half, so that both values
// of a pair are one lane's.  (Lanes copy 16 bytes in a row in either case.)
template <int D, bool kInterleaved>
struct RowPiece {
  static __device__ __forceinline__ uint4 load(const uint4* row, int sub) {  // in shared memory
    if constexpr (kInterleaved) return row[sub];
    const uint2 p = reinterpret_cast<const uint2*>(row)[sub], q = reinterpret_cast<const uint2*>(row)[D / 8 + sub];
    return make_uint4(p.x, p.y, q.x, q.y);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* row, int sub, const uint4& v) {
    if constexpr (kInterleaved) {
      *reinterpret_cast<uint4*>(row + sub * 8) = v;
    } else {
      *reinterpret_cast<uint2*>(row + sub * 4) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(row + D / 2 + sub * 4) = make_uint2(v.z, v.w);
    }
  }
  static __device__ __forceinline__ void weights(const float* w, int sub, float (&f)[8]) {
    const float4 p = __ldg(reinterpret_cast<const float4*>(w + (kInterleaved ? sub * 8 : sub * 4)));
    const float4 q = __ldg(reinterpret_cast<const float4*>(w + (kInterleaved ? sub * 8 + 4 : D / 2 + sub * 4)));
    f[0] = p.x; f[1] = p.y; f[2] = p.z; f[3] = p.w;
    f[4] = q.x; f[5] = q.y; f[6] = q.z; f[7] = q.w;
  }
};

// Rotation of a lane's four pairs.
template <int D, bool kInterleaved>
struct Rotation {
  float c[4], s[4];
  // t: the cos row, then the sin row, in shared memory
  __device__ __forceinline__ void load(const float4* t, int sub) {
    const float4 x = t[sub], y = t[D / 8 + sub];
    c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
    s[0] = y.x; s[1] = y.y; s[2] = y.z; s[3] = y.w;
  }
  __device__ __forceinline__ void scale(float r) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] *= r;
      s[k] *= r;
    }
  }
  __device__ __forceinline__ void apply(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float& a = f[kInterleaved ? 2 * k : k];
      float& b = f[kInterleaved ? 2 * k + 1 : k + 4];
      const float p = a, q = b;
      a = p * c[k] - q * s[k];
      b = p * s[k] + q * c[k];
    }
  }
};

// Copy of a table row: lanes below D / 8 take cos, as many behind them sin.
template <int D>
__device__ __forceinline__ void copy_table(const NormRopeArgs& a, int pos, uint4* to, int lane) {
  constexpr int kLanes = D / 8;
  if (lane < 2 * kLanes) {
    const int row = pos < 0 || pos >= a.n_pos ? 0 : pos;  // reported when the token comes
    const float* t = (lane < kLanes ? a.cos_t : a.sin_t) + int64_t(row) * (D / 2) + (lane % kLanes) * 4;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + lane)), "l"(t) : "memory");
  }
}

// A token of the cache is refused whole where its position is out of range, its value
// too; in the dense layout values have no positions.
__device__ __forceinline__ bool has_position(const NormRopeArgs& a, int side) { return a.cos_t && (side < 2 || a.slots); }

// Where the rows of a token go: out + h * step, `write` false where it must not.
struct RopePlace {
  __nv_bfloat16* out;
  int64_t step;
  bool write;
};
template <int D>
__device__ __forceinline__ RopePlace rope_place(const NormRopeArgs& a, int side, int token, int b, int pos, int slot,
                                                int lane) {
  RopePlace r{a.out[side], 0, true};
  const int H = a.heads[side];
  if (a.slots) {
    const int id = slot >> a.page_shift, page = 1 << a.page_shift;
    r.write = slot >= 0 && id < a.num_pages;
    if (slot >= 0 && !r.write && lane == 0) raise_error(AB_ERR_CAPACITY);
    r.out += side == 0 ? int64_t(token) * H * D : (int64_t(id) * H * page + (slot & (page - 1))) * D;
    r.step = side == 0 ? D : page * D;
  } else {
    const int len = a.len[side];
    r.out += (int64_t(b) * (H - 1) * len + token) * D;  // row (b H + h) len + t, token b len + t
    r.step = int64_t(len) * D;
  }
  if (has_position(a, side) && (pos < 0 || pos >= a.n_pos)) {
    if (r.write && lane == 0) raise_error(AB_ERR_CAPACITY);
    r.write = false;
  }
  return r;
}

// norm 0 and 1: a warp per unit.
template <int D, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 5) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  using Piece = RowPiece<D, kInterleaved>;
  constexpr int NV = kRopeRows, STAGES = kRopeStages;
  constexpr int kLanes = D / 8;       // lanes of a head row
  constexpr int kRows = 32 / kLanes;  // head rows a warp covers at once
  constexpr int kWarps = kRopeThreads / 32;
  extern __shared__ uint4 rope_smem[];  // [STAGES][NV][threads], [STAGES][threads], [STAGES][warps]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % kLanes, rsub = lane / kLanes;
  uint4* const pieces = rope_smem + threadIdx.x;
  uint4* const tables = rope_smem + STAGES * NV * kRopeThreads + warp * 32;
  int4* const places = reinterpret_cast<int4*>(rope_smem + STAGES * (NV + 1) * kRopeThreads) + warp;
  pdl_wait();
  pdl_trigger();
  const int n_units = a.n_units, step = int(gridDim.x) * kWarps;

  // What a unit is, read a unit ahead: x position, y slot, z token,
  // w side | group << 2 | batch element << 12 (B H <= 2^20).
  auto read_place = [&](int n) {
    int4 p = make_int4(0, 0, 0, 0);
    if (n < n_units) {
      int side, group;
      if (a.merged) {
        p.z = int(uint32_t(n) / uint32_t(a.units[2]));
        const int local = n - p.z * a.units[2];
        side = local < a.units[0] ? 0 : local < a.units[1] ? 1 : 2;
        group = local - (side == 0 ? 0 : a.units[side - 1]);
      } else {
        side = n < a.units[0] ? 0 : n < a.units[1] ? 1 : 2;
        const int first = side == 0 ? 0 : a.units[side - 1], local = n - first;
        const int groups = (a.units[side] - first) / a.tokens[side];
        p.z = int(uint32_t(local) / uint32_t(groups));
        group = local - p.z * groups;
      }
      const int b = a.len[side] == a.tokens[side] ? 0 : int(uint32_t(p.z) / uint32_t(a.len[side]));
      p.w = side | group << 2 | b << 12;
      if (has_position(a, side)) p.x = a.pos[side] ? __ldg(a.pos[side] + p.z) : p.z - b * a.len[side];
      if (a.slots) p.y = __ldg(a.slots + p.z);
    }
    return p;
  };

  // copies ahead: one step each, a unit's first step with its table row and place
  int ahead = blockIdx.x * kWarps + warp, left = 0, h_ahead = 0, H_ahead = 0;
  const __nv_bfloat16* src = nullptr;
  int64_t src_step = 0;
  int4 place = read_place(ahead);
  auto copy_next = [&](int stage) {
    if (left == 0 && ahead < n_units) {  // a unit begins
      const int side = place.w & 3, b = int(uint32_t(place.w) >> 12);
      const TokenView& x = a.in[side];
      left = a.steps[side];
      H_ahead = a.heads[side];
      h_ahead = ((place.w >> 2) & 1023) * left * (NV * kRows) + rsub;
      src = x.ptr + sub * 8 + b * x.sb + (place.z - b * a.len[side]) * x.st + h_ahead * x.sh;
      src_step = kRows * x.sh;
      if (side < 2 && a.cos_t) copy_table<D>(a, place.x, tables + stage * kRopeThreads, lane);
      if (lane == 0) places[stage * kWarps] = place;
      ahead += step;
      place = read_place(ahead);
    }
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h_ahead < H_ahead) cp_async16(smem_u32(pieces + (stage * NV + i) * kRopeThreads), src);
        h_ahead += kRows;
        src += src_step;
      }
      --left;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) copy_next(k);

  Rotation<D, kInterleaved> rot;
  float wv[8];
  int side = -1, todo = 0, h = 0, H = 0;
  int64_t out_step = 0;
  __nv_bfloat16* out = nullptr;
  bool write = false, rotate = false, weigh = false;
  int stage = 0;
  for (int n = blockIdx.x * kWarps + warp; n < n_units || todo > 0;) {
    __syncwarp();  // the warp is done with the stage that is filled next
    copy_next(stage == 0 ? STAGES - 1 : stage - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    if (todo == 0) {  // a unit begins
      const int4 p = places[stage * kWarps];
      const int cur = p.w & 3;
      todo = a.steps[cur];
      H = a.heads[cur];
      h = ((p.w >> 2) & 1023) * todo * (NV * kRows) + rsub;
      const RopePlace r = rope_place<D>(a, cur, p.z, int(uint32_t(p.w) >> 12), p.x, p.y, lane);
      write = r.write;
      out = r.out + h * r.step;
      out_step = kRows * r.step;
      rotate = cur < 2 && a.cos_t;
      if (rotate) rot.load(reinterpret_cast<const float4*>(tables + stage * kRopeThreads), sub);
      if (kNorm && cur < 2 && cur != side) {
        weigh = a.w[cur] != nullptr;
        if (weigh) Piece::weights(a.w[cur], sub, wv);
      }
      side = cur;
      n += step;
    }
    const uint4* in = pieces + stage * NV * kRopeThreads;
    if (side == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h < H && write) *reinterpret_cast<uint4*>(out + sub * 8) = in[i * kRopeThreads];
        h += kRows;
        out += out_step;
      }
    } else {
      uint4 x[NV];
      float r[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = Piece::load(in + i * kRopeThreads - sub, sub);  // of a head there is not: what is left there
        r[i] = kNorm ? sum_squares8(x[i]) : 1.f;
      }
      if constexpr (kNorm) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < NV; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i] = rsqrtf(fmaf(r[i], 1.f / float(D), a.eps));
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        widen8(x[i], f);
        if (kNorm && weigh) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= wv[k];
        }
        if (rotate) rot.apply(f);
        if constexpr (kNorm) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= r[i];
        }
        if (h < H && write) Piece::store(out, sub, round8(f));
        h += kRows;
        out += out_step;
      }
    }
    --todo;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// norm 2: a CTA per token.  NV head rows a lane, STAGES tokens in flight.
template <int D, bool kInterleaved, int NV, int STAGES>
__global__ void __launch_bounds__(640) token_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  using Piece = RowPiece<D, kInterleaved>;
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  extern __shared__ uint4 rope_smem[];  // as above
  __shared__ __align__(16) float part[2][16];
  const int threads = blockDim.x, warps = threads >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % kLanes, h0 = warp * kRows + lane / kLanes, hstep = warps * kRows;
  uint4* const pieces = rope_smem + threadIdx.x;
  uint4* const tables = rope_smem + STAGES * NV * threads + warp * 32;
  int4* const places = reinterpret_cast<int4*>(rope_smem + STAGES * (NV + 1) * threads) + warp;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) part[threadIdx.x >> 4][threadIdx.x & 15] = 0.f;
  __syncthreads();
  const int n_units = a.n_units, step = int(gridDim.x);

  // a token of the list: x position, y slot, z token, w side | batch element << 2
  auto read_place = [&](int n) {
    int4 p = make_int4(0, 0, 0, 0);
    if (n < n_units) {
      const int side = n < a.units[0] ? 0 : n < a.units[1] ? 1 : 2;
      p.z = n - (side == 0 ? 0 : a.units[side - 1]);
      const int b = a.len[side] == a.tokens[side] ? 0 : int(uint32_t(p.z) / uint32_t(a.len[side]));
      p.w = side | b << 2;
      if (has_position(a, side)) p.x = a.pos[side] ? __ldg(a.pos[side] + p.z) : p.z - b * a.len[side];
      if (a.slots) p.y = __ldg(a.slots + p.z);
    }
    return p;
  };
  int ahead = blockIdx.x;
  int4 place = read_place(ahead);
  auto copy_next = [&](int stage) {
    if (ahead < n_units) {
      const int side = place.w & 3, b = place.w >> 2, H = a.heads[side];
      const TokenView& x = a.in[side];
      const __nv_bfloat16* src = x.ptr + sub * 8 + b * x.sb + (place.z - b * a.len[side]) * x.st + h0 * x.sh;
      const int64_t next = hstep * x.sh;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h0 + i * hstep < H) cp_async16(smem_u32(pieces + (stage * NV + i) * threads), src);
        src += next;
      }
      if (side < 2 && a.cos_t) copy_table<D>(a, place.x, tables + stage * threads, lane);
      if (lane == 0) places[stage * warps] = place;
    }
    ahead += step;
    place = read_place(ahead);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) copy_next(k);

  float wv[NV][8], inv = 0.f;
  int side = -1, stage = 0, flip = 0;
  for (int n = blockIdx.x; n < n_units; n += step) {
    __syncwarp();
    copy_next(stage == 0 ? STAGES - 1 : stage - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const int4 p = places[stage * warps];
    const int cur = p.w & 3, H = a.heads[cur];
    if (cur < 2 && cur != side) {
      inv = 1.f / float(H * D);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) wv[i][k] = 1.f;
        if (a.w[cur] && h0 + i * hstep < H) Piece::weights(a.w[cur] + int64_t(h0 + i * hstep) * D, sub, wv[i]);
      }
    }
    side = cur;
    const RopePlace to = rope_place<D>(a, cur, p.z, p.w >> 2, p.x, p.y, lane);
    __nv_bfloat16* out = to.out + h0 * to.step;
    const int64_t out_step = hstep * to.step;
    const uint4* in = pieces + stage * NV * threads;
    if (cur == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h0 + i * hstep < H && to.write) *reinterpret_cast<uint4*>(out + sub * 8) = in[i * threads];
        out += out_step;
      }
    } else {
      const bool rotate = a.cos_t != nullptr;
      uint4 x[NV];
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = h0 + i * hstep < H ? Piece::load(in + i * threads - sub, sub) : make_uint4(0u, 0u, 0u, 0u);
        q += sum_squares8(x[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane == 0) part[flip][warp] = q;
      Rotation<D, kInterleaved> rot;
      if (rotate) rot.load(reinterpret_cast<const float4*>(tables + stage * threads), sub);
      __syncthreads();
      q = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k * 4 >= warps) break;
        const float4 y = reinterpret_cast<const float4*>(part[flip])[k];
        q += (y.x + y.y) + (y.z + y.w);
      }
      flip ^= 1;
      const float r = rsqrtf(fmaf(q, inv, a.eps));
      if (rotate) rot.scale(r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (warp * kRows + i * hstep >= H) break;
        float f[8];
        widen8(x[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= wv[i][k];
        if (rotate) {
          rot.apply(f);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= r;
        }
        if (h0 + i * hstep < H && to.write) Piece::store(out, sub, round8(f));
        out += out_step;
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

}  // namespace ab
