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
// into shared memory (cp.async) several units ahead, the token's table rows
// with them, and registers hold only the weights.  A unit is one token and the
// head rows that a warp covers in a step (norm 0 and 1), or one token and all
// heads, taken by a whole CTA (norm 2).  The units of q, k and v form one list
// that the CTAs walk together, so that the cheap ones (v is only moved) even
// out: token by token where a warp takes a unit (a fused projection is then
// read front to back), tensor by tensor where a CTA does and keeps a tensor's
// weights in registers.  Runs of 8 tokens are taken at about the same time, so
// that a head's output, rows of 128 or 256 bytes that lie a sequence apart, is
// written in longer pieces.  The factor r of a token's norm goes into its cos and sin once.
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
  const int32_t* pos[2];   // positions of q's and k's tokens, null: the token's index
  const float *cos_t, *sin_t;  // [n_pos, d/2], both null: no rotation
  int n_pos;
  float eps;
  int heads[3];
  int len[3];              // tokens per batch element
  int tokens[3];           // tokens in all
  int units[3];            // end of each one's units in the list; if merged, of each one's units within a token
  int groups[3];           // units of a token
  bool merged;             // token by token (all three have the same tokens, tokens_all)
  int tokens_all, n_units;
  int run_shift;           // log2 of the tokens of a run
  // paged destination
  const int32_t* slots;    // [T], null: the dense destination
  int page_shift, num_pages;
};

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

// Threads of a warp-per-unit CTA; head rows a lane takes per unit and units in
// flight (a CTA-per-token launch with many heads takes 8 rows and 2 units).
constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4, kRopeStages = 3;
constexpr int kRopeRowsMany = 8, kRopeStagesMany = 2;

// Bytes of shared memory: the pieces, the table rows and the place per warp.
__host__ __device__ constexpr int rope_smem_bytes(int nv, int stages, int threads) {
  return stages * threads * 16 * (nv + 1) + stages * (threads / 32) * 16;
}

// NV: head rows a lane takes per unit.  STAGES: units in flight.
template <int D, int NORM, bool kInterleaved, int NV, int STAGES>
__global__ void __launch_bounds__(NORM == kNormToken ? 640 : kRopeThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr bool kTeam = NORM == kNormToken;    // the CTA takes a token
  constexpr int kLanes = D / 8;                 // lanes of a head row
  constexpr int kRows = 32 / kLanes;            // head rows a warp covers at once
  constexpr int kPairs = kInterleaved ? 4 : 8;  // table entries of a lane
  extern __shared__ uint4 rope_smem[];          // [STAGES][NV][threads], [STAGES][threads], [STAGES][warps]
  const int threads = blockDim.x, warps = threads >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % kLanes, rsub = lane / kLanes;
  uint4* const pieces = rope_smem + threadIdx.x;
  uint4* const tables = rope_smem + STAGES * NV * threads + warp * 32;
  int4* const places = reinterpret_cast<int4*>(rope_smem + STAGES * (NV + 1) * threads) + warp;

  const int n_units = a.n_units;
  // a CTA that takes whole tokens takes runs of them
  const int run_mask = kTeam ? (1 << a.run_shift) - 1 : 0;
  const int step = kTeam ? int(gridDim.x) << a.run_shift : int(gridDim.x) * warps;
  auto next_unit = [&](int n) { return (n & run_mask) != run_mask ? n + 1 : n + step - run_mask; };
  // What a unit is, worked out once, ahead of its copies: x position, y slot,
  // z token, w side | group << 2 | batch element << 12 (B H <= 2^20).
  auto read_place = [&](int n) {
    int4 p = make_int4(0, 0, 0, 0);
    if (n < n_units) {
      int side, group;
      if (!kTeam && a.merged) {
        // runs of tokens, the units of a token, all runs
        const int per_run = a.units[2] << a.run_shift;
        const int run = int(uint32_t(n) / uint32_t(per_run));
        const int local = (n - run * per_run) >> a.run_shift;
        p.z = (run << a.run_shift) + (n & ((1 << a.run_shift) - 1));
        side = p.z >= a.tokens_all ? 3 : local < a.units[0] ? 0 : local < a.units[1] ? 1 : 2;
        group = local - (side == 0 ? 0 : a.units[side - 1]);
      } else {
        side = n < a.units[0] ? 0 : n < a.units[1] ? 1 : 2;
        p.z = n - (side == 0 ? 0 : a.units[side - 1]);
        group = 0;
        if (!kTeam) {
          const int local = p.z;
          p.z = int(uint32_t(local) / uint32_t(a.groups[side]));
          group = local - p.z * a.groups[side];
        }
      }
      p.w = side;
      if (side == 3) return p;  // behind the last token of a run
      const int b = a.len[side] == a.tokens[side] ? 0 : int(uint32_t(p.z) / uint32_t(a.len[side]));
      p.w |= group << 2 | b << 12;
      if (side < 2 && a.cos_t) p.x = a.pos[side] ? __ldg(a.pos[side] + p.z) : p.z - b * a.len[side];
      if (a.slots) p.y = __ldg(a.slots + p.z);
    }
    return p;
  };
  // first head row of this lane in a unit, further ones hstep apart
  auto head0 = [&](int4 p) { return (kTeam ? warp : ((p.w >> 2) & 1023) * NV) * kRows + rsub; };
  const int hstep = kTeam ? warps * kRows : kRows;

  auto issue = [&](int n, int4 p, int stage) {
    if (n < n_units && (p.w & 3) == 3) {
      if (lane == 0) places[stage * warps] = p;
    } else if (n < n_units) {
      const int side = p.w & 3, b = int(uint32_t(p.w) >> 12);
      const TokenView& x = a.in[side];
      const int H = a.heads[side];
      int h = head0(p);
      const __nv_bfloat16* src = x.ptr + sub * 8 + b * x.sb + (p.z - b * a.len[side]) * x.st + h * x.sh;
      const int64_t next = hstep * x.sh;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h < H) cp_async16(smem_u32(pieces + (stage * NV + i) * threads), src);
        h += hstep;
        src += next;
      }
      if (side < 2 && a.cos_t && lane < 2 * kLanes) {
        const int row = p.x < 0 || p.x >= a.n_pos ? 0 : p.x;  // reported when the unit comes
        const float* t = (lane < kLanes ? a.cos_t : a.sin_t) + int64_t(row) * (D / 2) + sub * 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(tables + stage * threads + lane)), "l"(t)
                     : "memory");
      }
      if (lane == 0) places[stage * warps] = p;
    }
    cp_async_commit();
  };

  int n = kTeam ? int(blockIdx.x) << a.run_shift : int(blockIdx.x) * warps + warp;
  int ahead = n;
  int4 place = read_place(ahead);
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) {
    issue(ahead, place, k);
    ahead = next_unit(ahead);
    place = read_place(ahead);
  }

  auto widen = [](const uint4& v, float (&f)[8]) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(x[k] << 16);
      f[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u);
    }
  };

  __shared__ float part[2][20];
  constexpr int kW = kTeam ? NV : 1;
  float wv[kW][8];  // weights of this lane, for all units of a side
  int side = -1;
  for (int stage = 0, flip = 0; n < n_units; n = next_unit(n)) {
    __syncwarp();  // the warp is done with the stage that is filled next
    issue(ahead, place, stage == 0 ? STAGES - 1 : stage - 1);
    ahead = next_unit(ahead);
    place = read_place(ahead);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint4* in = pieces + stage * NV * threads;
    const int4 here = places[stage * warps];
    const int cur = here.w & 3;
    if (cur == 3) {
      stage = stage == STAGES - 1 ? 0 : stage + 1;
      continue;
    }
    const int H = a.heads[cur];
    if (NORM != kNormNone && cur != side && cur < 2) {
      const float* w = a.w[cur];
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const int h = kTeam ? head0(here) + i * hstep : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) wv[i][k] = 1.f;
        if (w && h < H) {
          const float4* from = reinterpret_cast<const float4*>(w + int64_t(h) * D + sub * 8);
          const float4 p = __ldg(from), q = __ldg(from + 1);
          wv[i][0] = p.x; wv[i][1] = p.y; wv[i][2] = p.z; wv[i][3] = p.w;
          wv[i][4] = q.x; wv[i][5] = q.y; wv[i][6] = q.z; wv[i][7] = q.w;
        }
      }
      side = cur;
    }

    // destination row of head h: out + h * head_step
    const bool rotate = cur < 2 && a.cos_t != nullptr;
    bool write = true;
    __nv_bfloat16* out = a.out[cur] + sub * 8;
    int64_t head_step;
    if (a.slots) {
      const int id = here.y >> a.page_shift, page = 1 << a.page_shift;
      write = here.y >= 0 && id < a.num_pages;
      if (here.y >= 0 && !write && lane == 0) raise_error(AB_ERR_CAPACITY);
      out += cur == 0 ? int64_t(here.z) * H * D : (int64_t(id) * H * page + (here.y & (page - 1))) * D;
      head_step = cur == 0 ? D : page * D;
    } else {
      const int b = int(uint32_t(here.w) >> 12), len = a.len[cur];
      out += (int64_t(b) * (H - 1) * len + here.z) * D;  // row (b H + h) len + t, token b len + t
      head_step = int64_t(len) * D;
    }
    if (rotate && (here.x < 0 || here.x >= a.n_pos)) {
      if (write && lane == 0) raise_error(AB_ERR_CAPACITY);
      write = false;
    }
    int h = head0(here);
    out += h * head_step;
    head_step *= hstep;

    if (cur == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h < H && write) *reinterpret_cast<uint4*>(out) = in[i * threads];
        h += hstep;
        out += head_step;
      }
    } else {
      float c[kPairs], s[kPairs];
      if (rotate) {
        const float4* t = reinterpret_cast<const float4*>(tables + stage * threads);
#pragma unroll
        for (int k = 0; k < kPairs / 4; ++k) {
          const int at = kInterleaved ? sub : (sub % (kLanes / 2)) * 2 + k;
          const float4 x = t[at], y = t[kLanes + at];
          c[4 * k] = x.x; c[4 * k + 1] = x.y; c[4 * k + 2] = x.z; c[4 * k + 3] = x.w;
          s[4 * k] = y.x; s[4 * k + 1] = y.y; s[4 * k + 2] = y.z; s[4 * k + 3] = y.w;
        }
        // of a pair (i, i + d/2) the first becomes a cos - b sin, the second b cos + a sin
        if (!kInterleaved && sub < kLanes / 2) {
#pragma unroll
          for (int k = 0; k < kPairs; ++k) s[k] = -s[k];
        }
      }
      uint4 x[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = h + i * hstep < H ? in[i * threads] : make_uint4(0u, 0u, 0u, 0u);
      float r = 1.f;
      if constexpr (kTeam) {
        float q0 = 0.f, q1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          square_add(x[i].x, q0);
          square_add(x[i].y, q1);
          square_add(x[i].z, q0);
          square_add(x[i].w, q1);
        }
        float q = q0 + q1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
        if (lane == 0) part[flip][warp] = q;
        __syncthreads();
        q = 0.f;
        for (int k = 0; k < warps; ++k) q += part[flip][k];
        flip ^= 1;
        r = rsqrtf(q / float(H * D) + a.eps);
        if (rotate) {
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            c[k] *= r;
            s[k] *= r;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (h - rsub >= H) break;  // whole warps leave together: the shuffles below need every lane
        if constexpr (NORM == kNormHead) {
          float q0 = 0.f, q1 = 0.f;
          square_add(x[i].x, q0);
          square_add(x[i].y, q1);
          square_add(x[i].z, q0);
          square_add(x[i].w, q1);
          float q = q0 + q1;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          r = rsqrtf(fmaf(q, 1.f / float(D), a.eps));
        }
        float f[8];
        widen(x[i], f);
        if constexpr (NORM != kNormNone) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= wv[kTeam ? i : 0][k];
        }
        if (rotate) {
          if constexpr (kInterleaved) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float p = f[2 * k], q = f[2 * k + 1];
              f[2 * k] = p * c[k] - q * s[k];
              f[2 * k + 1] = p * s[k] + q * c[k];
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float o = __shfl_xor_sync(0xffffffffu, f[k], kLanes / 2);
              f[k] = f[k] * c[k] + o * s[k];
            }
          }
        }
        if (NORM == kNormHead || (kTeam && !rotate)) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= r;
        }
        if (h < H && write)
          *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                     pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        h += hstep;
        out += head_step;
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

}  // namespace ab
