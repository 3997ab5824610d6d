// Page layout and decode of the MXFP4 latent cache, shared by its writer (norm_rope.hip), its
// reader (latent_gather.hip) and the attention over it (attn_paged.hip).
//
// A page holds 64 tokens: 64 code rows of latent / 2 bytes (element 2j in the low nibble of byte
// j), then 64 scale rows of latent / 32 bytes (UE8M0, one a block of 32 values), then 64
// positional rows of 64 bf16 values.  All three begin at multiples of 128 bytes.
#pragma once

#include "common.hpp"

namespace mxidx {

constexpr int kLatentRope = 64;            // positional values of a latent row

template <int kLatent>
struct MxPage {
  static constexpr int kCodes = kLatent / 2, kScales = kLatent / kBlock, kPos = kLatentRope * 2;   // a row's bytes
  static constexpr int kScaleBase = kPage * kCodes, kPosBase = kScaleBase + kPage * kScales;
  static constexpr int kBytes = kPosBase + kPage * kPos;
  static_assert(kScaleBase % 128 == 0 && kPosBase % 128 == 0 && kBytes % 128 == 0, "aligned parts");
};

constexpr int mx_page_bytes(int latent) { return kPage * (latent / 2 + latent / kBlock + kLatentRope * 2); }

// 2^(s - 127) of a scale byte s, as the conversions take it: they read the exponent's bits alone, 0
// among them as 2^-127.
__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(s << 23); }

// 8 codes (a dword) to 8 bf16 values, exact: two significant bits times a power of two from
// 2^-127 on, whose smallest half-steps are subnormal and still a bf16.
__device__ __forceinline__ uint4 mx_decode8(uint32_t codes, float scale) {
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3)));
}

}  // namespace mxidx
