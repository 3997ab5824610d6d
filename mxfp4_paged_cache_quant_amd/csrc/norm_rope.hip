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
// whole wave (256: 32 lanes, 128: 16), a positional part of 64 eight lanes; the
// sums of a row are xor-shuffles over its lanes.  Bound by HBM: each value is read
// and written once.
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

template <int W>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int m = 1; m < W; m <<= 1) s += __shfl_xor(s, m, W);
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
  const float r = 1.0f / sqrtf(row_sum<W>(s) * inv_n + eps);
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

template <bool kF32>
__global__ __launch_bounds__(256) void norm_rope_kernel(HeadsSpec q, HeadsSpec k, int64_t rows,
                                                        RopeSpec rs) {
  const int sub = threadIdx.x & 15;
  const int heads = q.heads + k.heads;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 4);
  for (int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4; row < rows; row += step) {
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    const HeadsSpec& s = h < q.heads ? q : k;
    const int hh = h < q.heads ? h : h - q.heads;
    float v[8], w[8], b[8];
    load8<kF32>(s.x, t * s.row_stride + hh * s.head_stride + 8 * sub, v);
    load_params(s.weight, sub, 1.f, w);
    load_params(s.bias, sub, 0.f, b);
    norm_row8<16>(v, s.norm, s.eps, w, b);
    if (rs.rope_dim > 0) rope_row8<16>(v, sub, rs.positions ? rs.positions[t] : t, rs);
    store8<kF32>(s.out, t * s.out_row_stride + hh * s.out_head_stride + 8 * sub, v);
  }
}

// Blocks [0, q_blocks) rotate the query rows, 8 lanes a row; the others take one
// token per wave: kLatent / 8 lanes norm the latent part, the first 8 rotate the rest.
template <bool kF32, int kLatent>
__global__ __launch_bounds__(256) void latent_insert_kernel(LatentSpec a, RopeSpec rs, int q_blocks) {
  if ((int)blockIdx.x < q_blocks) {
    const int sub = threadIdx.x & (kRopeLanes - 1);
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kRopeLanes;
    if (row >= a.T * a.H) return;
    const int64_t t = row / a.H;
    const int64_t h = row - t * a.H;
    float v[8];
    load8<kF32>(a.q_pe, t * a.q_row_stride + h * a.q_head_stride + 8 * sub, v);
    rope_row8<kRopeLanes>(v, sub, rs.positions ? rs.positions[t] : t, rs);
    store8<false>(a.q_out, t * a.out_row_stride + h * a.out_head_stride + 8 * sub, v);
    return;
  }
  constexpr int W = kLatent / 8;
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = ((int64_t)(blockIdx.x - q_blocks) * blockDim.x + threadIdx.x) / kWave;
  if (t >= a.T) return;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0 || slot >= a.num_slots) return;        // uniform over the wave
  const int64_t src = t * a.kv_row_stride, dst = slot * (kLatent + kRopeWidth);
  float v[8], w[8], b[8];
  if (lane < W) {
    load8<kF32>(a.kv, src + 8 * lane, v);
    load_params(a.weight, lane, 1.f, w);
    load_params(nullptr, lane, 0.f, b);
    norm_row8<W>(v, a.norm, a.eps, w, b);
    store8<false>(a.cache, dst + 8 * lane, v);
  }
  if (lane < kRopeLanes) {
    load8<kF32>(a.kv, src + kLatent + 8 * lane, v);
    rope_row8<kRopeLanes>(v, lane, rs.positions ? rs.positions[t] : t, rs);
    store8<false>(a.cache, dst + kLatent + 8 * lane, v);
  }
}

template <bool kF32>
hipError_t launch_latent(const LatentSpec& a, int latent, const RopeSpec& rs, hipStream_t stream) {
  const int64_t q_rows = a.q_pe ? a.T * a.H : 0;
  const int q_blocks = (int)((q_rows * kRopeLanes + 255) / 256);
  const int blocks = q_blocks + (int)((a.T * kWave + 255) / 256);
  switch (latent) {
    case 128:
      hipLaunchKernelGGL((latent_insert_kernel<kF32, 128>), dim3(blocks), dim3(256), 0, stream, a, rs, q_blocks);
      break;
    case 256:
      hipLaunchKernelGGL((latent_insert_kernel<kF32, 256>), dim3(blocks), dim3(256), 0, stream, a, rs, q_blocks);
      break;
    default:
      hipLaunchKernelGGL((latent_insert_kernel<kF32, 512>), dim3(blocks), dim3(256), 0, stream, a, rs, q_blocks);
      break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(const HeadsSpec& q, const HeadsSpec& k, bool f32, int64_t T,
                            const RopeSpec& rope, hipStream_t stream) {
  const int64_t rows = T * (q.heads + k.heads);
  const int64_t blocks = (rows + 15) / 16;
  const int grid = (int)(blocks < 256 * 32 ? blocks : 256 * 32);
  if (f32)
    hipLaunchKernelGGL(norm_rope_kernel<true>, dim3(grid), dim3(256), 0, stream, q, k, rows, rope);
  else
    hipLaunchKernelGGL(norm_rope_kernel<false>, dim3(grid), dim3(256), 0, stream, q, k, rows, rope);
  return hipGetLastError();
}

hipError_t launch_latent_insert(const LatentSpec& a, bool f32, int latent, const RopeSpec& rope,
                                hipStream_t stream) {
  return f32 ? launch_latent<true>(a, latent, rope, stream)
             : launch_latent<false>(a, latent, rope, stream);
}

}  // namespace mxidx
