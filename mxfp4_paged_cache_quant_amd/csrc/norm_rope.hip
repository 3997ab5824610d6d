// Per-head norm and rotary position embedding in one pass: the indexer's query and
// key rows (idx_norm_rope), and the main cache's latent rows with their paged write
// and the query's positional part (idx_latent_insert).
//
// Norm of a row of n values, in fp32:
//   rms:   y = x * rsqrt(sum x^2 / n + eps) * weight + bias
//   layer: the same of x - m, m = sum x / n (the mean subtracted before squaring, so
//          a mean that is large beside the spread loses nothing)
// then the rotation of rope.hpp, then one rounding to the output's type.
//
// Work mapping: 8 values a lane, so a row of 128 is 16 lanes, a latent row of 512 a
// whole wave (256: 32 lanes, 128: 16), a positional part of 64 eight lanes.  The lanes of
// a row keep to one token for a run of its heads: angles and weights are loaded once a
// run, and kBatch rows are loaded ahead of their arithmetic.  The sums go round rings
// of 16 lanes (no LDS), the root is the hardware's reciprocal one, and the rotation's
// sign is in the angles.
//
// Bound by HBM: each value is read and written once.  8192 tokens of 65 heads, bf16:
// 63.6 us, 4.3 TB/s where a large copy makes 4.9 (a row at a time, with its angles and
// weights -- six times its bytes from the first cache --, a 64-bit division and shuffled
// sums: 105 us; the runs alone: 75).  16384 tokens of 576 values and 32 query heads of
// 64: 39.9 us, 4.4 TB/s (45.9 before the runs).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "rope.hpp"

namespace mxidx {
namespace {

constexpr int kRopeLanes = 8;              // lanes of a 64-value positional part
constexpr int kRopeWidth = 64;

template <bool kF32>
__device__ __forceinline__ void load8(const void* base, int64_t off, float (&v)[8]) {
  if constexpr (kF32) {
    const float* p = static_cast<const float*>(base) + off;
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

// Two fp32 values to bf16, round to nearest even (a in the low half).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

template <bool kF32>
__device__ __forceinline__ void store8(void* base, int64_t off, const float (&v)[8]) {
  if constexpr (kF32) {
    float* p = static_cast<float*>(base) + off;
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7]));
  }
}

// x of the lane n places on in its row of 16 lanes (the row taken as a ring).
template <int n>
__device__ __forceinline__ float ring16(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + n, 0xf, 0xf, true));
}

// The sum over a row's W lanes, in each of them (every sum is of two equal halves, so all
// lanes get the same bits).
template <int W>
__device__ __forceinline__ float row_sum(float s) {
  static_assert(W >= 16, "whole rings");
  s += ring16<8>(s);
  s += ring16<4>(s);
  s += ring16<2>(s);
  s += ring16<1>(s);
#pragma unroll
  for (int m = 16; m < W; m <<= 1) s += __shfl_xor(s, m);
  return s;
}

// The norm of a row of 8W values held by W lanes (w, b: this lane's 8 weights).
template <int W>
__device__ __forceinline__ void norm_row8(float (&v)[8], int norm, float eps, const float (&w)[8],
                                          const float (&b)[8]) {
  if (norm == kNormNone) return;
  constexpr float inv_n = 1.0f / (8 * W);
  if (norm == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
    const float m = row_sum<W>(s) * inv_n;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] -= m;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += v[i] * v[i];
  const float r = rsqrtf(row_sum<W>(s) * inv_n + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i] + b[i];
}

__device__ __forceinline__ void load_params(const float* p, int sub, float other, float (&v)[8]) {
  if (p) {
    load8<true>(p, 8 * sub, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = other;
  }
}

constexpr int kBatch = 4;     // rows loaded together where runs are long enough

// Runs of run_len heads of one token, 16 lanes each: all of q's runs, then all of k's.
template <bool kF32, int kRun>
__global__ __launch_bounds__(256) void norm_rope_kernel(HeadsSpec q, HeadsSpec k, uint32_t q_units,
                                                        uint32_t units, int run_len, RopeSpec rs) {
  const int sub = threadIdx.x & 15;
  uint32_t unit = (blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  if (unit >= units) return;                         // uniform over a row's lanes
  const bool is_q = unit < q_units;
  const HeadsSpec& s = is_q ? q : k;
  if (!is_q) unit -= q_units;
  const uint32_t runs = (uint32_t)(s.heads + run_len - 1) / (uint32_t)run_len;
  const uint32_t t = unit / runs;
  const int h0 = (int)(unit - t * runs) * run_len, h1 = min(h0 + run_len, s.heads);
  const int64_t src = t * s.row_stride + 8 * sub, dst = t * s.out_row_stride + 8 * sub;
  RopeAngles angles;
  if (rs.rope_dim > 0) rope_angles(angles, sub, rs.positions ? rs.positions[t] : t, rs);
  float w[8], b[8];
  load_params(s.weight, sub, 1.f, w);
  load_params(s.bias, sub, 0.f, b);
  for (int h = h0; h < h1; h += kRun) {
    float v[kRun][8];
#pragma unroll
    for (int i = 0; i < kRun; ++i)                   // past the run: its last row again
      load8<kF32>(s.x, src + min(h + i, h1 - 1) * s.head_stride, v[i]);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      norm_row8<16>(v[i], s.norm, s.eps, w, b);
      if (rs.rope_dim > 0) rotate_row8<16>(v[i], sub, angles, rs);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (h + i < h1) store8<kF32>(s.out, dst + (h + i) * s.out_head_stride, v[i]);
  }
}

// Blocks [0, q_blocks) rotate the query rows, 8 lanes for a run of heads of one token; the
// others take kTokens tokens a wave: kLatent / 8 lanes norm the latent part, the first
// 8 rotate the rest.
template <bool kF32, int kLatent, int kTokens, int kRun>
__global__ __launch_bounds__(256) void latent_insert_kernel(LatentSpec a, RopeSpec rs, int q_blocks,
                                                            int run_len) {
  if ((int)blockIdx.x < q_blocks) {
    const int sub = threadIdx.x & (kRopeLanes - 1);
    const uint32_t unit = (blockIdx.x * blockDim.x + threadIdx.x) / kRopeLanes;
    const uint32_t runs = (uint32_t)(a.H + run_len - 1) / (uint32_t)run_len;
    const uint32_t t = unit / runs;
    if (t >= a.T) return;
    const int h0 = (int)(unit - t * runs) * run_len, h1 = min(h0 + run_len, a.H);
    const int64_t src = t * a.q_row_stride + 8 * sub, dst = t * a.out_row_stride + 8 * sub;
    RopeAngles angles;
    rope_angles(angles, sub, rs.positions ? rs.positions[t] : t, rs);
    for (int h = h0; h < h1; h += kRun) {
      float v[kRun][8];
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        load8<kF32>(a.q_pe, src + min(h + i, h1 - 1) * a.q_head_stride, v[i]);
#pragma unroll
      for (int i = 0; i < kRun; ++i) rotate_row8<kRopeLanes>(v[i], sub, angles, rs);
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (h + i < h1) store8<false>(a.q_out, dst + (h + i) * a.out_head_stride, v[i]);
    }
    return;
  }
  constexpr int W = kLatent / 8;
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t first = ((int64_t)(blockIdx.x - q_blocks) * blockDim.x + threadIdx.x) / kWave * kTokens;
  const int wl = lane < W ? lane : 0, rl = lane & (kRopeLanes - 1);   // lanes without a part read another's
  float w[8], b[8];
  load_params(a.weight, wl, 1.f, w);
  load_params(nullptr, wl, 0.f, b);
  int64_t slot[kTokens];
  float v[kTokens][8], r[kTokens][8];
  RopeAngles angles[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = min(first + i, a.T - 1);
    slot[i] = first + i < a.T ? a.slot_mapping[t] : -1;
    load8<kF32>(a.kv, t * a.kv_row_stride + 8 * wl, v[i]);
    load8<kF32>(a.kv, t * a.kv_row_stride + kLatent + 8 * rl, r[i]);
    rope_angles(angles[i], rl, rs.positions ? rs.positions[t] : t, rs);
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    norm_row8<W>(v[i], a.norm, a.eps, w, b);
    rotate_row8<kRopeLanes>(r[i], rl, angles[i], rs);
    if (slot[i] < 0 || slot[i] >= a.num_slots) continue;
    const int64_t dst = slot[i] * (kLatent + kRopeWidth);
    if (lane < W) store8<false>(a.cache, dst + 8 * lane, v[i]);
    if (lane < kRopeLanes) store8<false>(a.cache, dst + kLatent + 8 * lane, r[i]);
  }
}

// Heads of a run: kBatch rows or more while the call has lanes enough to fill the card
// (256 CUs of 2048), one otherwise.
int run_length(int64_t rows, int lanes) {
  int n = 4 * kBatch;
  while (n >= kBatch && rows * lanes / n < 256 * 2048) n /= 2;
  return n >= kBatch ? n : 1;
}

// `many`: the call fills the card with runs of kBatch rows and two tokens a wave.
template <bool kF32, int kLatent>
void launch_latent_rows(const LatentSpec& a, const RopeSpec& rs, int q_blocks, int run_len, bool many,
                        hipStream_t stream) {
  const int64_t waves = many ? (a.T + 1) / 2 : a.T;
  const dim3 grid((uint32_t)(q_blocks + (waves + 3) / 4));
  if (many)
    hipLaunchKernelGGL((latent_insert_kernel<kF32, kLatent, 2, kBatch>), grid, dim3(256), 0, stream, a, rs,
                       q_blocks, run_len);
  else
    hipLaunchKernelGGL((latent_insert_kernel<kF32, kLatent, 1, 1>), grid, dim3(256), 0, stream, a, rs,
                       q_blocks, run_len);
}

template <bool kF32>
hipError_t launch_latent(const LatentSpec& a, int latent, const RopeSpec& rs, hipStream_t stream) {
  const bool many = a.T >= 2 * 256 * 32 || (a.q_pe && run_length(a.T * a.H, kRopeLanes) > 1);
  const int run_len = many && a.q_pe ? std::max(run_length(a.T * a.H, kRopeLanes), kBatch) : 1;
  const int64_t units = a.q_pe ? a.T * ((a.H + run_len - 1) / run_len) : 0;
  const int q_blocks = (int)((units * kRopeLanes + 255) / 256);
  switch (latent) {
    case 128: launch_latent_rows<kF32, 128>(a, rs, q_blocks, run_len, many, stream); break;
    case 256: launch_latent_rows<kF32, 256>(a, rs, q_blocks, run_len, many, stream); break;
    default: launch_latent_rows<kF32, 512>(a, rs, q_blocks, run_len, many, stream); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(const HeadsSpec& q, const HeadsSpec& k, bool f32, int64_t T,
                            const RopeSpec& rope, hipStream_t stream) {
  const int run_len = run_length(T * (q.heads + k.heads), 16);
  const uint32_t q_units = (uint32_t)(T * ((q.heads + run_len - 1) / run_len));
  const uint32_t units = q_units + (uint32_t)(T * ((k.heads + run_len - 1) / run_len));
  const dim3 grid((units + 15) / 16);
#define MXIDX_NORM(f32_, run)                                                                      \
  hipLaunchKernelGGL((norm_rope_kernel<f32_, run>), grid, dim3(256), 0, stream, q, k, q_units, units, \
                     run_len, rope)
  if (run_len == 1) {
    if (f32) MXIDX_NORM(true, 1); else MXIDX_NORM(false, 1);
  } else {
    if (f32) MXIDX_NORM(true, kBatch); else MXIDX_NORM(false, kBatch);
  }
#undef MXIDX_NORM
  return hipGetLastError();
}

hipError_t launch_latent_insert(const LatentSpec& a, bool f32, int latent, const RopeSpec& rope,
                                hipStream_t stream) {
  return f32 ? launch_latent<true>(a, latent, rope, stream)
             : launch_latent<false>(a, latent, rope, stream);
}

}  // namespace mxidx
