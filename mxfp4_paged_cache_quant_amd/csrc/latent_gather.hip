// MXFP4 latent cache -> contiguous bf16 rows (idx_latent_gather_mxfp4): the cached contexts of a
// prefill, read back in token order.
//
// One workgroup of four waves takes a (sequence, page): latent / 8 lanes decode a token's codes,
// 8 values (a dword) a lane, so that a wave's stores are whole rows; eight lanes copy its
// positional part.  kBatch of a wave's rows are loaded before the first is written.
//
// Bound by HBM, mostly by its writes (400 B read and 1152 B written a token at latent 512): 122,880
// tokens of eight requests 43.3 us = 4.4 TB/s, where a large copy makes 4.7-4.9; 110,000 tokens of
// 200 requests, latent 128, 13.6 us = 4.7 TB/s.
#include "common.hpp"
#include "latent_mxfp4.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

template <int kLatent>
__global__ __launch_bounds__(256) void latent_gather_kernel(LatentGatherArgs a) {
  using Page = MxPage<kLatent>;
  constexpr int W = kLatent / 8, kAt = kWave / W;        // lanes of a row, rows of a wave at a time
  constexpr int kRows = kPage / 4;                       // of a wave
  constexpr int kBatch = kRows / kAt < 8 ? kRows / kAt : 8;
  const int b = blockIdx.y;
  const int64_t lp = blockIdx.x;                         // logical page of sequence b
  const int64_t len = min((int64_t)a.seq_lens[b], a.max_seq_len);
  const int64_t page = a.block_table[b * a.bt_row_stride + lp], first = a.cu_seq_offsets[b] + lp * kPage;
  if (page < 0 || page >= a.num_pages) return;
  // the page's tokens that there are, and that have a row
  const int n = (int)max(min(len - lp * kPage, (int64_t)kPage), (int64_t)0);
  const int r0 = first < 0 ? (int)min(-first, (int64_t)kPage) : 0;
  const int r1 = (int)min((int64_t)n, max(a.total_tokens - first, (int64_t)0));
  if (r1 <= r0) return;
  const uint8_t* src = a.cache + page * Page::kBytes;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + first * a.out_row_stride;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int sub = lane % W, t0 = wave * kRows + lane / W;
#pragma unroll
  for (int i = 0; i < kRows / kAt; i += kBatch) {
    uint32_t codes[kBatch], scale[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = t0 + (i + j) * kAt;                  // in the page, whether it holds a token or not
      codes[j] = *reinterpret_cast<const uint32_t*>(src + t * Page::kCodes + 4 * sub);
      scale[j] = src[Page::kScaleBase + t * Page::kScales + sub / 4];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = t0 + (i + j) * kAt;
      if (t >= r0 && t < r1)
        *reinterpret_cast<uint4*>(dst + t * a.out_row_stride + 8 * sub) = mx_decode8(codes[j], mx_scale(scale[j]));
    }
  }
  constexpr int kPosRows = kWave / 8;                    // positional rows of a wave at a time
#pragma unroll
  for (int i = 0; i < kRows; i += kPosRows) {
    const int t = wave * kRows + i + lane / 8;
    if (t >= r0 && t < r1)
      *reinterpret_cast<uint4*>(dst + t * a.out_row_stride + kLatent + 8 * (lane % 8)) =
          *reinterpret_cast<const uint4*>(src + Page::kPosBase + t * Page::kPos + 16 * (lane % 8));
  }
}

}  // namespace

hipError_t launch_latent_gather(const LatentGatherArgs& a, int latent, hipStream_t stream) {
  const dim3 grid((unsigned)((a.max_seq_len + kPage - 1) / kPage), (unsigned)a.batch);
  switch (latent) {
    case 128: hipLaunchKernelGGL((latent_gather_kernel<128>), grid, dim3(256), 0, stream, a); break;
    case 256: hipLaunchKernelGGL((latent_gather_kernel<256>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((latent_gather_kernel<512>), grid, dim3(256), 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace mxidx
