// Rotary position embedding of a row held 8 values to a lane, shared by the query
// encoders (insert.hip) and the norm + rotation kernels (norm_rope.hip).
//
// The pairs (j, j + rope_dim/2) (neox) or (2j, 2j+1) (interleaved) are rotated by
// angle j:  a' = a*cos - b*sin,  b' = b*cos + a*sin, each product and each sum
// rounded to fp32 (no fused multiply-add), so the rotated values are exactly
// defined.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace mxidx {

__device__ __forceinline__ float rot_a(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return a * c - b * s;
}
__device__ __forceinline__ float rot_b(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return b * c + a * s;
}

// The angles that a lane of a row needs (lane sub of W holding values 8sub..8sub+7), for
// kernels that rotate several rows by the same ones.  Neox: v' = v*c + partner*s with s
// negated for the first half, which rounds as a*c - b*s does.
struct RopeAngles {
  float c[8], s[8];          // interleaved: the first 4
  bool on;                   // this lane's values are rotated
};

// Angles of table row p: rope_dim is a multiple of 16, at most 8W, so each lane's 8 values
// are all rotated or all not; a position outside the table rotates nothing.
__device__ __forceinline__ void rope_angles(RopeAngles& a, int sub, int64_t p, const RopeSpec& rs) {
  const int half = rs.rope_dim >> 1, hl = half >> 3;
  a.on = p >= 0 && p < rs.table_rows && sub < (rs.rope_dim >> 3);
  if (!a.on) return;
  const bool low = sub < hl;
  const int j0 = rs.interleaved ? 4 * sub : 8 * (low ? sub : sub - hl);
  const float* cr = rs.cos_t + p * half + j0;
  const float* sr = rs.sin_t + p * half + j0;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (rs.interleaved && i > 0) break;
    const float4 c = *reinterpret_cast<const float4*>(cr + i);
    const float4 s = *reinterpret_cast<const float4*>(sr + i);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a.c[i + j] = cc[j];
      a.s[i + j] = low && !rs.interleaved ? -ss[j] : ss[j];
    }
  }
}

// Rotates the row that W lanes hold by those angles.  A neox lane's partners sit in one
// other lane of the row (lane sub +- rope_dim/16) and come by shuffles, so every lane of
// the row calls it.
template <int W>
__device__ __forceinline__ void rotate_row8(float (&v)[8], int sub, const RopeAngles& a, const RopeSpec& rs) {
#pragma clang fp contract(off)
  if (rs.interleaved) {
    if (!a.on) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = rot_a(x, y, a.c[i], a.s[i]);
      v[2 * i + 1] = rot_b(x, y, a.c[i], a.s[i]);
    }
    return;
  }
  const int hl = rs.rope_dim >> 4, partner = sub < hl ? sub + hl : sub - hl;
  float pv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) pv[i] = __shfl(v[i], partner, W);
  if (!a.on) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * a.c[i] + pv[i] * a.s[i];
}

// Rotates the row that 16 lanes hold (lane sub: elements 8sub..8sub+7) by the
// angles of table row p; a position outside the table leaves it unrotated.
// Every lane of the row calls it: a neox lane's partners come by shuffles.
__device__ __forceinline__ void rope_row8(float (&v)[8], int sub, int64_t p, const RopeSpec& rs) {
  const int half = rs.rope_dim >> 1;
  const int hl = half >> 3;                     // lanes per half of the rotated range
  const bool ok = p >= 0 && p < rs.table_rows;  // same for the row's 16 lanes
  float pv[8];
  if (!rs.interleaved) {
    const int partner = sub < hl ? sub + hl : sub - hl;
#pragma unroll
    for (int i = 0; i < 8; ++i) pv[i] = __shfl(v[i], partner, 16);
  }
  if (!ok || sub >= (rs.rope_dim >> 3)) return;
  const float* cr = rs.cos_t + p * half;
  const float* sr = rs.sin_t + p * half;
  if (rs.interleaved) {
    // pairs (8sub + 2i, 8sub + 2i + 1), angle index 4sub + i
    const float4 c = *reinterpret_cast<const float4*>(cr + 4 * sub);
    const float4 s = *reinterpret_cast<const float4*>(sr + 4 * sub);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = rot_a(a, b, cc[i], ss[i]);
      v[2 * i + 1] = rot_b(a, b, cc[i], ss[i]);
    }
  } else {
    // this lane holds elements 8sub..8sub+7: the a's of angles 8sub.. (sub < hl)
    // or the b's of angles 8(sub - hl).. ; the partner lane holds the others
    const int j0 = 8 * (sub < hl ? sub : sub - hl);
    const float4 c0 = *reinterpret_cast<const float4*>(cr + j0);
    const float4 c1 = *reinterpret_cast<const float4*>(cr + j0 + 4);
    const float4 s0 = *reinterpret_cast<const float4*>(sr + j0);
    const float4 s1 = *reinterpret_cast<const float4*>(sr + j0 + 4);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (sub < hl) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = rot_a(v[i], pv[i], cc[i], ss[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = rot_b(pv[i], v[i], cc[i], ss[i]);
    }
  }
}

}  // namespace mxidx
