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
// Bound by memory: 2 bytes in and 2 bytes out per value against about 12
// operations.  One CTA takes one token of one of q, k, v, so that a token's
// table row is read by one SM and its heads share it; a head's d values lie in
// d / 8 lanes of 16 bytes, so every access is a whole head row (128 or 256
// bytes), and each lane issues all of its loads before it uses the first.
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
  int first_block[3];      // first CTA of each of the three (k's and v's; q's is 0)
  // paged destination
  const int32_t* slots;    // [T], null: the dense destination
  int page_shift, num_pages;
};

constexpr int kRopeVecs = 8;  // head rows per lane at most

template <int D, int NORM, bool kInterleaved>
__global__ void __launch_bounds__(512) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int kLanes = D / 8;           // lanes of a head row
  constexpr int kRows = 32 / kLanes;      // head rows a warp covers at once
  constexpr int kPairs = kInterleaved ? 4 : 8;  // table entries of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int sub = lane % kLanes;
  int side = 0;
  if (int(blockIdx.x) >= a.first_block[2]) side = 2;
  else if (int(blockIdx.x) >= a.first_block[1]) side = 1;
  const int token = int(blockIdx.x) - (side == 0 ? 0 : a.first_block[side]);
  const int len = a.len[side], H = a.heads[side];
  const int b = token / len, t = token - b * len;
  const bool work = side < 2;

  // destination row of head h: out + h * head_step
  __nv_bfloat16* out = a.out[side];
  int64_t head_step;
  if (a.slots) {
    const int slot = __ldg(a.slots + token);
    if (slot < 0) return;  // padding
    if (slot >> a.page_shift >= a.num_pages) {
      if (threadIdx.x == 0) raise_error(AB_ERR_CAPACITY);
      return;
    }
    if (side == 0) {
      out += int64_t(token) * H * D;
      head_step = D;
    } else {
      const int page = 1 << a.page_shift;
      out += ((int64_t(slot >> a.page_shift) * H * page) + (slot & (page - 1))) * D;
      head_step = int64_t(page) * D;
    }
  } else {
    out += (int64_t(b) * H * len + t) * D;
    head_step = int64_t(len) * D;
  }

  const bool rotate = work && a.cos_t != nullptr;
  int pos = t;
  if (rotate) {
    if (a.pos[side]) pos = __ldg(a.pos[side] + token);
    if (pos < 0 || pos >= a.n_pos) {
      if (threadIdx.x == 0) raise_error(AB_ERR_CAPACITY);
      return;
    }
  }

  const __nv_bfloat16* in = a.in[side].ptr + int64_t(b) * a.in[side].sb + int64_t(t) * a.in[side].st + sub * 8;
  const int64_t sh = a.in[side].sh;
  const int h0 = warp * kRows + lane / kLanes, hstep = warps * kRows;
  uint4 x[kRopeVecs];
#pragma unroll
  for (int i = 0; i < kRopeVecs; ++i) {
    const int h = h0 + i * hstep;
    if (h < H) x[i] = __ldcs(reinterpret_cast<const uint4*>(in + h * sh));
  }
  if (!work) {
#pragma unroll
    for (int i = 0; i < kRopeVecs; ++i) {
      const int h = h0 + i * hstep;
      if (h < H) *reinterpret_cast<uint4*>(out + h * head_step + sub * 8) = x[i];
    }
    return;
  }

  float c[kPairs], s[kPairs];
  if (rotate) {
    const int first = kInterleaved ? sub * 4 : (sub % (kLanes / 2)) * 8;
    const float4* pc = reinterpret_cast<const float4*>(a.cos_t + int64_t(pos) * (D / 2) + first);
    const float4* ps = reinterpret_cast<const float4*>(a.sin_t + int64_t(pos) * (D / 2) + first);
#pragma unroll
    for (int k = 0; k < kPairs / 4; ++k) {
      const float4 u = __ldg(pc + k), v = __ldg(ps + k);
      c[4 * k] = u.x; c[4 * k + 1] = u.y; c[4 * k + 2] = u.z; c[4 * k + 3] = u.w;
      s[4 * k] = v.x; s[4 * k + 1] = v.y; s[4 * k + 2] = v.z; s[4 * k + 3] = v.w;
    }
    // the second of a pair (i, i + d/2) gets a sin + b cos: fold the sign in
    if (!kInterleaved && sub < kLanes / 2)
#pragma unroll
      for (int k = 0; k < kPairs; ++k) s[k] = -s[k];
  }

  auto widen = [](const uint4& v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  };

  const float* w = a.w[side];
  float r = 1.f;
  if constexpr (NORM == kNormToken) {
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeVecs; ++i) {
      if (h0 + i * hstep < H) {
        float f[8];
        widen(x[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) q = fmaf(f[k], f[k], q);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    __shared__ float part[16];
    if (lane == 0) part[warp] = q;
    __syncthreads();
    q = 0.f;
    for (int k = 0; k < warps; ++k) q += part[k];
    r = 1.f / sqrtf(q / float(H * D) + a.eps);
  }
  float wv[8];
  auto load_w = [&](const float* from) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(from)), v = __ldg(reinterpret_cast<const float4*>(from) + 1);
    wv[0] = u.x; wv[1] = u.y; wv[2] = u.z; wv[3] = u.w;
    wv[4] = v.x; wv[5] = v.y; wv[6] = v.z; wv[7] = v.w;
  };
  if (NORM == kNormHead && w) load_w(w + sub * 8);

#pragma unroll
  for (int i = 0; i < kRopeVecs; ++i) {
    const int h = h0 + i * hstep;
    if (h - lane / kLanes >= H) break;  // whole warps leave together: the shuffles below need every lane
    const bool on = h < H;
    float f[8];
    if (!on) x[i] = make_uint4(0u, 0u, 0u, 0u);
    widen(x[i], f);
    if constexpr (NORM == kNormHead) {
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) q = fmaf(f[k], f[k], q);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      r = 1.f / sqrtf(q * (1.f / float(D)) + a.eps);
    }
    if constexpr (NORM != kNormNone) {
      if (NORM == kNormToken && w && on) load_w(w + int64_t(h) * D + sub * 8);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = w ? f[k] * r * wv[k] : f[k] * r;
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
    if (on)
      *reinterpret_cast<uint4*>(out + h * head_step + sub * 8) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

}  // namespace ab
