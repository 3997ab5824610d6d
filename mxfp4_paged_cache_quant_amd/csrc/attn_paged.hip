// Attention over the paged latent cache (idx_attn_paged): for each query row r and
// head h, with row_j the cached row of visible token j and n the latent size,
//   s_j = scale * sum_i q[r,h,i] * row_j[i]  (n + 64 values),
//   out[r,h,:] = sum_j exp(s_j - m) * row_j[:n] / l,  l = sum_j exp(s_j - m),
//   lse[r,h] = m + log l,  m = max_j s_j.
//
// One pass over the tokens with the running maximum and sum: a new maximum scales what
// was summed so far by exp(m_old - m_new).  One workgroup per (row, head); its four waves
// take every fourth token each, 64 lanes sharing a row's values, and join at the end.
#include "common.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

constexpr int kRopeWidth = 64;
constexpr int kWaves = 4;

__device__ __forceinline__ float bf16_to_f32(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// The cache row of entry j of query row r, or -1 where there is none.
__device__ __forceinline__ int64_t token_row(const AttnArgs& a, int64_t r, int64_t j, int seq,
                                             int64_t ks, int64_t window) {
  int64_t p = j;
  if (a.indices) p = (int64_t)a.indices[r * a.idx_row_stride + j] - ks;
  if (p < 0 || p >= window) return -1;
  const int page = a.block_table[seq * a.bt_row_stride + p / kPage];
  if (page < 0 || page >= a.num_pages) return -1;
  return (int64_t)page * kPage + p % kPage;
}

template <int kLatent>
__global__ __launch_bounds__(kWaves * kWave) void attn_simple_kernel(AttnArgs a) {
  constexpr int kRow = kLatent + kRopeWidth;
  constexpr int kPer = kRow / kWave, kOut = kLatent / kWave;
  __shared__ float part[kWaves][kLatent];
  __shared__ float part_m[kWaves], part_l[kWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t r = blockIdx.x / a.H;
  const int h = (int)(blockIdx.x % a.H);
  const int seq = a.row_seq ? a.row_seq[r] : (int)(r / a.rows_per_seq);
  if (seq < 0 || seq >= a.B) return;
  const int64_t ks = a.ks ? a.ks[r] : 0;
  const int64_t window = min(max((int64_t)a.ke[r] - ks, (int64_t)0), a.max_tokens);
  const int64_t entries = a.indices ? a.k : window;

  const uint16_t* q = static_cast<const uint16_t*>(a.q) + r * a.q_row_stride + h * a.q_head_stride;
  float qv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) qv[i] = bf16_to_f32(q[lane + i * kWave]);
  float m = neg_inf(), l = 0.f, o[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) o[i] = 0.f;
  for (int64_t j = wave; j < entries; j += kWaves) {
    const int64_t row = token_row(a, r, j, seq, ks, window);
    if (row < 0) continue;
    const uint16_t* c = static_cast<const uint16_t*>(a.cache) + row * kRow;
    float kv[kPer], s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) kv[i] = bf16_to_f32(c[lane + i * kWave]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) s += qv[i] * kv[i];
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) s += __shfl_xor(s, x);
    s *= a.scale;
    const float m2 = fmaxf(m, s);
    const float old = m2 == m ? 1.f : expf(m - m2), p = s == m2 ? 1.f : expf(s - m2);
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < kOut; ++i) o[i] = o[i] * old + p * kv[i];
    m = m2;
  }
#pragma unroll
  for (int i = 0; i < kOut; ++i) part[wave][lane + i * kWave] = o[i];
  if (lane == 0) {
    part_m[wave] = m;
    part_l[wave] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  float mm = neg_inf(), ll = 0.f, f[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, part_m[w]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    f[w] = part_l[w] == 0.f ? 0.f : expf(part_m[w] - mm);
    ll += f[w] * part_l[w];
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + r * a.out_row_stride + h * a.out_head_stride;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += f[w] * part[w][lane + i * kWave];
    out[lane + i * kWave] = f32_to_bf16(ll == 0.f ? 0.f : v / ll);
  }
  if (a.lse && lane == 0) a.lse[r * a.H + h] = ll == 0.f ? neg_inf() : mm + logf(ll);
}

}  // namespace

int64_t attn_workspace_bytes(int64_t, int, int, int64_t) { return 0; }

hipError_t launch_attn_paged(const AttnArgs& a, int latent, void*, hipStream_t stream) {
  const dim3 grid((uint32_t)(a.rows * a.H)), block(kWaves * kWave);
  switch (latent) {
    case 128: hipLaunchKernelGGL(attn_simple_kernel<128>, grid, block, 0, stream, a); break;
    case 256: hipLaunchKernelGGL(attn_simple_kernel<256>, grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL(attn_simple_kernel<512>, grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace mxidx
