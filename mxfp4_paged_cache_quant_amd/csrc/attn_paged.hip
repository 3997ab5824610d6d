// Attention over the paged latent cache (idx_attn_paged; in MXFP4, idx_attn_paged_mxfp4): for each query row r and
// head h, with row_j the cached row of visible token j and n the latent size,
//   s_j = scale * sum_i q[r,h,i] * row_j[i]  (n + 64 values),
//   out[r,h,:] = sum_j exp(s_j - m) * row_j[:n] / l,  l = sum_j exp(s_j - m),
//   lse[r,h] = m + log l,  m = max_j s_j.
//
// One pass over the tokens with the running maximum and sum (in powers of two): a
// new maximum scales what was summed so far by 2^(m_old - m_new).
//
// Work mapping: one workgroup takes HG * 16 heads of one query row over one share of
// the row's tokens, 64 tokens (a tile; 32 for many rows of more than 32 heads) at a time.  A wave holds 16
// heads: their query in registers and their output sums, HG waves the heads and TH waves
// the tile's token parts.  All products run on the 16x16x32 bf16 MFMA in the transposed
// form:
//   S^T = K Q^T   A = 16 tokens of the tile, B = the wave's 16 heads
//   O^T = V^T P^T A = 16 of the n values over 32 tokens, B = the weights
// so a lane holds one head throughout: the weights leave the first product in the
// registers where the second takes them (lane group g: tokens 4g..4g+3 of two 16-token
// parts), and the running maximum and sum are one register each.
//
// A row serves as key and, in its first n values, as value, so each cached row is
// read once into LDS (two tiles, the next one's loads between the current one's
// products).  The copies go straight from the cache rows to LDS in 16-byte
// chunks; chunk c of token t lands at place c ^ swz(t) of the row, which spreads both
// the keys' reads (16 tokens, one chunk) and the values' transposing reads (16 tokens,
// two neighbouring chunks) over all banks.  The query comes the same way, once.
//
// What bounds it: with many rows the instruction issue of two waves a SIMD and LDS
// together (1024 rows x 2048 tokens x 64 heads: of the SIMDs' cycles 54% MFMAs and 30%
// other vector instructions, LDS 51% busy without a bank conflict), 363-383 us = 760-805
// TFLOP/s, the weights' second part not counted, where a large library product reaches 1,306;
// with few rows the way to the first tile (the row's window, its list, its pages, the rows:
// four round trips) and the partial sums.  32 heads a wave with the tile's weights passed
// through LDS halves the LDS reads, but not the instructions (with the weights in one part
// 8 waves 482 us, 4 waves of 512 registers 512 us, where this form took 367).  A vector register
// spilled in the loop is read back behind the copies on their way, so none may be (one part: 331
// us with 5 of them, 312 without).  Scalar ones go to lanes of a vector register, no memory: in the
// 16- and 32-head forms of latent 512 16 and 26 of them do, read back 0 and 11 times in two tiles.
// Below, pairs of figures of steps inside the loop are of one part on both sides.
//
// Places of a tile that hold no visible token read as zeros and get weight 0, so
// nothing that a masked place holds reaches a sum.
//
// The weights go to the second product in two bf16 parts, the rounded weight and what rounding
// left (2^-16 of it at most); l and lse take them unrounded.  The output's error is then its own
// rounding's whatever the call's sizes.  With one part (2^-8) it is 1.24 times that over 2048
// tokens, and a row that one token dominates is off by that token's rounding, since the
// reference is no power of two from it.  Two parts are half as many products again: 1024 rows of
// 2048 tokens, 64 heads, 322 -> 378 us; 32 windows of 6600, 128 heads, 90 -> 102; 64 rows of 2048,
// 128 heads, 74 -> 79; 16 rows of 2048, 64 heads, 24 -> 25.
//
// Few rows: the tokens are split over workgroups, each leaving its unscaled sums with
// m and l in the workspace, and a second launch joins them.
//
// Over the MXFP4 cache the tiles in LDS are the same bf16 ones, expanded once for all of a
// workgroup's heads, so that the products stay as they are: 4-bit products would need the query and the
// weights in 8 bits or fewer.  The codes come two tiles ahead into a third buffer, which fills the LDS,
// and each lane expands what it copied while the second product runs (kMx).  That is 32 conversions and
// 8 stores a wave and tile beside 100 MFMAs (64 heads): 1024 rows of 2048 tokens 387 us, 358-374
// over the bf16 cache; where HBM counts for more the smaller rows make up for it: 64 rows of 2048
// tokens, 128 heads, 68-72 us (70-74), 16 x 2 windows of 6600 107 (101-104), one row of 131072,
// 64 heads, 52.6 (57), 16 rows of 2048, 64 heads, 25.6 (24.6).  Steps: codes in registers a tile ahead
// (20 of them spilled) 476 us for the 1024 rows; copied to LDS two tiles ahead, 32-bit addresses and
// no spills 404; sixteen lanes' stores on all banks, and scales four a lane where registers lack, 387.
// Two things that are left cost no time.  The first of those stores waits for the positional rows' copies,
// which go to the same array; with arrays of their own that wait is gone and the 1024 rows take 386
// us, the windows 107, the 16 rows 25.5.  Of the LDS's busy cycles 17% are bank conflicts, a fifth of them
// of the codes' reads (lanes 16 apart); without those 394 and 393 us, 107 and 107.
// Beyond 4 GiB the copies of codes take 64-bit addresses, which only the flat form of a copy to LDS has for
// each lane, and the compiler's first wait in a step is then for all of them: 1024 rows of 2048 tokens, 64 heads 397 us
// over 5 GB and 371 over 1, 16 heads 291 and 234; 32 windows of 6600, 128 heads 99.6 and 95.
#include <algorithm>

#include "common.hpp"
#include "latent_mxfp4.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

constexpr int kRopeWidth = kLatentRope;
constexpr int kCus = 256;
constexpr int kMaxSplits = 128;
constexpr float kSlack = 8.f;               // weights stay below 2^8 of the reference's

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
#define MXIDX_LDS __attribute__((address_space(3)))
#define MXIDX_GLOBAL __attribute__((address_space(1)))

__device__ __forceinline__ v4f mfma_bf16(v8s a, v8s b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ float low_half(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_half(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// LDS place of a 16-byte chunk: chunk c of token t's row is stored at c ^ swz(t).
// Latent rows are multiples of 256 bytes, so their banks repeat every 16 chunks and swz
// runs over 16 values; the 8-token groups that one pass of a read takes (0..7 and 8..15
// for the transposing reads, which take chunk pairs, {0..3, 12..15} and the like for the
// 16-byte ones) fall on different places.  Measured: 4.0 cycles a
// 16-byte and 2.5 a transposing read of a wave, none lost; with the same values in plain
// order 8.0 and 2.5.  The 128-byte positional rows alternate between two halves of the
// banks, and 8 values over token pairs do (4.0 cycles).
template <int kChunks>
__device__ __forceinline__ int swz(int t) {
  if constexpr (kChunks >= 16) return (((t & 7) ^ (((t >> 3) & 1) << 2)) << 1) | ((t >> 3) & 1);
  return (t >> 1) & 7;
}

// The maximum over the four lanes of one head (lane groups of 16).
__device__ __forceinline__ float max_groups(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The lane number, computed anew where it is called: nothing derived from it can be
// kept in registers from one call to the next.
__device__ __forceinline__ int fresh_lane() {
  int zero = 0;
  asm volatile("" : "+v"(zero));
  return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, (uint32_t)zero));
}

struct Row {                               // a query row's window
  int seq;
  int ks;
  int window;
};

// False when the row belongs to no sequence.
__device__ __forceinline__ bool row_of(const AttnArgs& a, int64_t r, Row& o) {
  o.seq = a.row_seq ? a.row_seq[r] : (int)((uint32_t)r / (uint32_t)a.rows_per_seq);
  if (o.seq < 0 || o.seq >= a.B) return false;
  o.ks = a.ks ? a.ks[r] : 0;
  o.window = (int)min(max((int64_t)a.ke[r] - (int64_t)o.ks, (int64_t)0), a.max_tokens);
  return true;
}

// A lane's token of a tile, in the steps that the pipeline takes apart so that none
// waits for its load at once: the list entry (of a window: the place itself), the token
// of the sequence (-1: none), its page, and then its cache row.  Loads of places
// without a token read a token's that is there.
__device__ __forceinline__ int list_entry(const AttnArgs& a, int64_t r, int e) {
  return a.indices ? a.indices[r * a.idx_row_stride + min(e, a.k - 1)] : e;
}

__device__ __forceinline__ int token_of(const AttnArgs& a, const Row& row, int entry, int e) {
  if (!a.indices) return entry < row.window ? entry : -1;
  const uint32_t p = (uint32_t)entry - (uint32_t)row.ks;   // exact from ks on
  return entry >= row.ks && p < (uint32_t)row.window && e < a.k ? (int)p : -1;
}

__device__ __forceinline__ int token_page(const AttnArgs& a, const Row& row, int p) {
  return a.block_table[row.seq * a.bt_row_stride + max(p, 0) / kPage];
}

// Partial sums of the split form: for each (row, split) HP x n output sums, then
// (m, l) of each head; HP = heads rounded up to the workgroups' heads.
struct Parts {
  float* o;
  float* ml;
  int splits, heads;
  int pages;              // of the cache
  uint32_t cache_bytes;   // the cache's size where it is below 4 GiB, and of a query row's heads
  uint32_t q_bytes;
};

// 16 bytes a lane to LDS, at dst + 16 * lane.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t rs, MXIDX_LDS uint8_t* dst, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (MXIDX_LDS void*)dst, 16, (int)offset, 0, 0, 0);
}

// The copy of a tile's rows to LDS, kMine of them by each wave, in kPieces parts that
// the caller issues between its products: latent rows first, then the positional ones,
// C 16-byte chunks of each.  Lane t of `rows` holds token t's row: where 32-bit offsets
// reach the whole cache (kSmall) its byte there, and rows that fill less than an
// instruction share one; else its number (stride bytes each), with a descriptor for each
// row and both its parts behind one another (the parts in two passes, with a descriptor
// each: 84 us for 64 rows of 2048 tokens, 128 heads; 75 so).  A place without a row (kNoRow) is out of its descriptor's
// range and reads as zeros.
constexpr int64_t kReach = 0xfffe0000ll;   // of 32-bit offsets
constexpr int kNoRow = (int)0xffff0000u;   // past it, no wrap within a row

struct Source {
  const char* base;
  uint32_t bytes;         // kSmall: of the whole
  int64_t stride;         // else: from one row to the next
};

template <int kLatent, int kTile, int kMine, bool kSmall>
struct TileCopy {
  static constexpr int kRowBytes = (kLatent + kRopeWidth) * 2;
  static constexpr int LC = kLatent / 8, PC = kRopeWidth / 8;
  static constexpr int kLatentPer = LC >= kWave || !kSmall ? 1 : kWave / LC;
  static constexpr int kPosPer = kWave / PC;
  static constexpr int kLatentPieces = kMine / kLatentPer;
  static constexpr int kPieces = kLatentPieces + (kSmall ? kMine / kPosPer : 0);
  static_assert(kMine % kLatentPer == 0 && kMine % kPosPer == 0, "whole instructions");

  template <int C, int kPer>
  static __device__ __forceinline__ void part(const Source& src, MXIDX_LDS uint8_t* dst, int t0, int rows,
                                              int offset, int ln) {
    const int t = t0 + (kPer == 1 ? 0 : ln / C);
    const int row = kPer == 1 ? __builtin_amdgcn_readlane(rows, t) : __builtin_amdgcn_ds_bpermute(4 * t, rows);
    // unsigned: a row of a cache above 2 GiB may begin below 2^31 and end above
    copy16(buffer_rsrc(src.base, (int)src.bytes), dst + t0 * C * 16,
           (uint32_t)row + (uint32_t)offset + (uint32_t)(((ln % C) ^ swz<C>(t)) << 4));
  }

  // One row, its latent part and its positional one, from a descriptor of its own.
  static __device__ __forceinline__ void whole(const Source& src, MXIDX_LDS uint8_t* tile, int t, int rows,
                                               int ln) {
    asm volatile("" : "+s"(t));                        // what follows from it is not kept over the loop
    const int row = __builtin_amdgcn_readlane(rows, t);
    const __amdgpu_buffer_rsrc_t rs =
        buffer_rsrc(src.base + (uint32_t)row * src.stride, row == kNoRow ? 0 : kRowBytes);
    if (LC >= kWave || ln < LC) copy16(rs, tile + t * LC * 16, (ln << 4) ^ (swz<LC>(t) << 4));
    if (ln < PC)
      copy16(rs, tile + kTile * kLatent * 2 + t * PC * 16, ((ln << 4) ^ (swz<PC>(t) << 4)) + kLatent * 2);
  }

  // Piece i of the rows from `first` on.
  static __device__ __forceinline__ void piece(int i, const Source& src, MXIDX_LDS uint8_t* tile, int first,
                                               int rows, int ln) {
    if constexpr (!kSmall)
      whole(src, tile, first + i, rows, ln);
    else if (i < kLatentPieces)
      part<LC, kLatentPer>(src, tile, first + i * kLatentPer, rows, 0, ln);
    else
      part<PC, kPosPer>(src, tile + kTile * kLatent * 2, first + (i - kLatentPieces) * kPosPer, rows, kLatent * 2,
                        ln);
  }
};

// The same of a cache in MXFP4.  The wave's kMine code rows go straight to a buffer in LDS of their own,
// a block's 16 bytes a lane, two tiles ahead; each lane then takes what it copied, its block's scale
// in a register, to the next tile as bf16 while the second product runs.  The positional rows go
// straight to the tile.  Lane t of `rows` holds token t's row: where 32-bit offsets reach the whole cache
// (kSmall) its page's byte there, a multiple of 256, plus its place in the page; else its number.
// A place without a row is out of the descriptor's range and reads as zeros; in the other form it
// reads row 0's (there is one: a window over a cache without pages is empty) under the scale 1,
// so that its values are finite: its weight is 0, and a score of its positional part, whatever that
// holds, is masked.  That scale is put in where the codes are expanded (take): a choice at the load
// would wait for it, and for the copies issued with it, at once (a cache of 5 GB, 32 windows of 6600
// tokens, 128 heads: 104.4 us, 99.6 so; one row of 131072, 64 heads: 60.9 and 57.7).
template <int kLatent, int kTile, int kMine, bool kSmall, bool kSpare>
struct MxCopy {
  using Page = MxPage<kLatent>;
  using Bytes = MXIDX_GLOBAL const uint8_t*;
  static constexpr int LB = kLatent / kBlock, LC = kLatent / 8, PC = kRopeWidth / 8;
  static constexpr int kPer = kWave / LB, kLoads = (kMine + kPer - 1) / kPer;      // tokens a load
  static constexpr int kPosPer = kWave / PC, kPosPieces = kMine / kPosPer;
  static constexpr int kYoungest = kSpare ? 2 * kLoads : kLoads + 1;                // instructions of load()
  static constexpr int kRawBytes = kLoads * kWave * 16;                            // of the wave
  static constexpr int SD = LB / 4;                    // dwords of a token's scales
  static constexpr int kDwords = 4 * kLoads;           // a lane's
  static_assert(kMine % kPosPer == 0 && (kMine % kPer == 0 || kMine < kPer) && kMine * SD <= kWave, "whole instructions");
  static_assert(Page::kBytes % 256 == 0 && Page::kBytes < 65536, "a row's place fits its page's lowest bits");

  uint32_t scales[kSpare ? kLoads : 1], scale, codes[2];
  uint32_t from, to;

  static __device__ __forceinline__ int row_code(bool ok, uint32_t page, uint32_t place) {
    return !ok ? kNoRow : (int)(kSmall ? page * (uint32_t)Page::kBytes + place : page * kPage + place);
  }

  // The token, from `first` on, that a lane's part of load i belongs to (lanes past the last: its).
  static __device__ __forceinline__ int token(int i, uint32_t ln) {
    return kMine < kPer ? min((int)(ln / LB), kMine - 1) : i * kPer + (int)(ln / LB);
  }

  // Byte `at` of the row's part that begins at `part` of its page, `bytes` a row.
  static __device__ __forceinline__ uint32_t offset(int row, uint32_t bytes, uint32_t at) {
    const uint32_t place = (uint32_t)row & (kPage - 1);
    return ((uint32_t)row & ~(uint32_t)(kPage - 1)) + place * bytes + at;
  }
  static __device__ __forceinline__ Bytes address(Bytes cache, int row, uint32_t bytes, uint32_t at) {
    asm volatile("" : "+s"(cache));                    // added to the offset where it is: no copy of it kept in lanes
    const uint32_t r = row == kNoRow ? 0u : (uint32_t)row;
    return cache + (int64_t)(r / kPage) * Page::kBytes + ((r % kPage) * bytes + at);
  }

  // 16 bytes a lane to LDS, at dst + 16 * lane.
  static __device__ __forceinline__ void copy(const Source& src, int row, uint32_t bytes, uint32_t at,
                                              MXIDX_LDS uint8_t* dst) {
    if constexpr (kSmall)
      copy16(buffer_rsrc(src.base, (int)src.bytes), dst, offset(row, bytes, at));
    else
      __builtin_amdgcn_global_load_lds((MXIDX_GLOBAL void*)address((Bytes)src.base, row, bytes, at),
                                       (MXIDX_LDS void*)dst, 16, 0, 0);
  }

  // The scales and the codes.
  __device__ __forceinline__ void load(const Source& src, MXIDX_LDS uint8_t* raw, int first, int rows, uint32_t ln) {
    auto scale_at = [&](int row, uint32_t at) __attribute__((always_inline)) {
      if constexpr (kSmall) {
        const int o = (int)offset(row, Page::kScales, Page::kScaleBase + at);
        if constexpr (kSpare) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(buffer_rsrc(src.base, (int)src.bytes), o, 0, 0);
        else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(buffer_rsrc(src.base, (int)src.bytes), o, 0, 0);
      } else {
        const Bytes p = address((Bytes)src.base, row, Page::kScales, Page::kScaleBase + at);
        return kSpare ? (uint32_t)*p : *(MXIDX_GLOBAL const uint32_t*)p;
      }
    };
    if constexpr (!kSpare)
      scales[0] = scale_at(__builtin_amdgcn_ds_bpermute(4 * (first + min((int)(ln / SD), kMine - 1)), rows), 4 * (ln % SD));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = __builtin_amdgcn_ds_bpermute(4 * (first + token(i, ln)), rows);
      if constexpr (kSpare) scales[i] = scale_at(row, ln % LB);
      copy(src, row, Page::kCodes, 16 * (ln % LB), raw + i * (kWave * 16));
    }
  }

  static __device__ __forceinline__ void position(int i, const Source& src, MXIDX_LDS uint8_t* tile, int first,
                                                  int rows, uint32_t ln) {
    const int t0 = first + i * kPosPer, t = t0 + (int)(ln / PC);
    const int row = __builtin_amdgcn_ds_bpermute(4 * t, rows);
    copy(src, row, Page::kPos, Page::kPosBase + (((ln % PC) ^ (uint32_t)swz<PC>(t)) << 4),
         tile + kTile * kLatent * 2 + t0 * PC * 16);
  }

  // A lane's way from the buffer to the tile: it takes the dwords of its 16 bytes in an order of its own
  // (dword j ^ turn as the j-th), so that sixteen lanes' stores of 16 bytes fall on all banks.  The
  // tokens of load i differ from those of load 0 in bits of their own, and swz is linear in bits.
  __device__ __forceinline__ void prepare(int first, uint32_t ln) {
    const uint32_t c = ln % LB, turn = LB == 16 ? (ln >> 2) & 3 : LB == 8 ? (ln >> 2) & 1 : (ln >> 3) & 1;
    const int t = first + token(0, ln);
    from = 16 * ln + 4 * turn;
    to = (uint32_t)t * (kLatent * 2) + (((4 * c + turn) ^ (uint32_t)swz<LC>(t)) << 4);
  }

  // Dword u % 4 of load u / 4, and with a load's first one its block's scale.  Bit t of `there`: the wave's
  // token t has a row.
  __device__ __forceinline__ void take(int u, MXIDX_LDS const uint8_t* raw, uint32_t ln, uint32_t there) {
    if (!kSpare && u % 4 == 0) {
      const int four = __builtin_amdgcn_ds_bpermute(4 * (token(u / 4, ln) * SD + (int)(ln % LB / 4)), (int)scales[0]);
      scale = __builtin_amdgcn_ubfe((uint32_t)four, 8 * (ln % 4), 8);
    }
    if (!kSmall && u % 4 == 0) {
      uint32_t& s = kSpare ? scales[u / 4] : scale;
      s = (there >> token(u / 4, kSpare ? (uint32_t)fresh_lane() : ln)) & 1 ? s : 0x7fu;
    }
    codes[u % 2] = *(MXIDX_LDS const uint32_t*)(raw + (from ^ (4u * (u % 4))) + u / 4 * (kWave * 16));
  }

  __device__ __forceinline__ void write(int u, MXIDX_LDS uint8_t* tile) const {
    *(MXIDX_LDS v8s*)(tile + (to ^ (uint32_t)((swz<LC>(u / 4 * kPer) ^ (u % 4)) << 4)) + u / 4 * kPer * (kLatent * 2)) =
        __builtin_bit_cast(v8s, mx_decode8(codes[u % 2], mx_scale(kSpare ? scales[u / 4] : scale)));
  }
};

template <int kLatent, int kTile, int HG, int TH, bool kSmall, bool kMx>
__global__ __launch_bounds__(HG * TH * kWave, kTile == 32 ? 2 : 1) void attn_kernel(AttnArgs a, Parts parts) {
  constexpr int kRow = kLatent + kRopeWidth;
  constexpr int kWaves = HG * TH, kHeads = HG * 16;
  constexpr int kTokens = kTile / TH;                  // of a tile, per wave
  constexpr int NT = kTokens / 16;                     // 16-token parts of those
  static_assert(NT == 1 || NT == 2, "one step of the second product");
  constexpr int KS = kRow / 32, KL = kLatent / 32;     // contraction steps, latent ones
  constexpr int NV = kLatent / 16;                     // 16-value parts of the output
  constexpr int LC = kLatent / 8;                      // 16-byte chunks of a latent row
  constexpr int kAhead = kSmall && !(kMx && HG > 2) ? 3 : 2;        // operand steps in flight from LDS, as registers allow
  constexpr int kValuesAhead = HG <= 2 ? 4 : kAhead;
  constexpr int kMine = kTile / kWaves;                // rows that a wave copies
  constexpr int kLatentBytes = kTile * kLatent * 2, kTileBytes = kTile * kRow * 2;
  using Copy = TileCopy<kLatent, kTile, kMine, kSmall>;
  constexpr bool kSpare = HG <= 2;                     // registers: these forms have a SIMD's to a wave
  using Mx = MxCopy<kLatent, kTile, kMine, kSmall, kSpare>;
  // Two arrays, and the loop below unrolled over them: the compiler then sees that a
  // tile's reads do not touch the one being copied, and does not wait for its copies.
  __shared__ __attribute__((aligned(1024))) uint8_t tile0[kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t tile1[kTileBytes];
  static_assert(kTile <= kWave && 2 * kTileBytes <= 156 * 1024, "a lane for each token; two tiles fit the LDS");
  // kMx: the codes of a tile.  With latent 512 the three arrays are the whole LDS of a CU, or of half of one
  // with 32-token tiles, so that the waves' statistics take the codes' place in the end.
  constexpr int kStatBytes = TH * kHeads * (int)sizeof(float2);
  __shared__ __attribute__((aligned(1024))) uint8_t last[kMx ? kWaves * Mx::kRawBytes : kStatBytes];
  static_assert(sizeof(last) >= kStatBytes, "the statistics' place");
  float2(*stats)[kHeads] = reinterpret_cast<float2(*)[kHeads]>(last);   // the waves' (m, l)

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int hg = wave % HG, th = wave / HG;
  // Workgroups go to the eight XCDs in turn: each takes a run of neighbouring numbers, so that
  // the head groups of a row, and rows of one sequence, read the same rows through one L2 (16
  // rows of 2048 tokens, 2 groups: 27.3 -> 23.6 us; 64 rows of two: 86.6 -> 83.7)
  const uint32_t xcd = blockIdx.x % 8, number = xcd * (gridDim.x / 8) + min(xcd, gridDim.x % 8) + blockIdx.x / 8;
  const uint32_t groups = (uint32_t)parts.heads / kHeads, unit = number / groups;
  const int group = (int)(number - unit * groups);
  const uint32_t r32 = unit / (uint32_t)parts.splits;
  const int split = (int)(unit - r32 * (uint32_t)parts.splits);
  const int64_t r = r32;
  Row row;
  if (!row_of(a, r, row)) return;
  const int entries = row.window == 0 || (kMx && parts.pages == 0) ? 0 : a.indices ? a.k : row.window;
  const int tiles = (entries + kTile - 1) / kTile;
  const int share = tiles / parts.splits, more = tiles - share * parts.splits;
  const int t0 = split * share + min(split, more);     // the first `more` splits take one more
  const int t1 = t0 + share + (split < more ? 1 : 0);

  v8s q[KS];                                           // step s: values 32s + 8g .. +7
  v4f o[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) o[v] = v4f{0.f, 0.f, 0.f, 0.f};
  float m = neg_inf(), l = 0.f;                        // l: this lane's tokens only
  const float scale2 = a.scale * 1.4426950408889634f;  // scores in powers of two
  bool seen = false;                                   // a visible token

  // The lanes' cache rows of a tile, and which places hold a token.
  auto rows_of = [&](int p, int page, uint64_t& mask) __attribute__((always_inline)) {
    const bool ok = p >= 0 && page >= 0 && page < parts.pages;
    mask = __ballot(ok);
    if constexpr (kMx) return Mx::row_code(ok, (uint32_t)page, (uint32_t)p & (kPage - 1));
    const uint32_t row = (uint32_t)page * kPage + ((uint32_t)p & (kPage - 1));
    return ok ? (int)(kSmall ? row * (kRow * 2) : row) : kNoRow;
  };
  const Source cache{static_cast<const char*>(a.cache), parts.cache_bytes, kRow * 2};
  MXIDX_LDS uint8_t* raw = (MXIDX_LDS uint8_t*)last + wave * Mx::kRawBytes;
  Mx mx;                                               // kMx: the scales of the codes there

  // The wave's kTokens tokens of a tile against its heads; the pieces of the next tile's
  // copy go between the steps of the first product.
  auto compute = [&](MXIDX_LDS const uint8_t* buf, uint64_t mask, MXIDX_LDS uint8_t* nxt, int rows,
                     uint64_t next_mask) __attribute__((always_inline)) {
    const int base = th * kTokens;
    v4f s[NT];
    if constexpr (kMx) {
      const int ln = fresh_lane();
#pragma unroll
      for (int i = 0; i < Mx::kPosPieces; ++i) Mx::position(i, cache, nxt, wave * kMine, rows, ln);
      __builtin_amdgcn_sched_barrier(0);
    }
    {
      // LDS offsets of the operands in the tile: the places of the chunks differ
      // between steps by constants xored into few bits (swz), so one register for each
      // kind of row does
      const int ln = fresh_lane(), n = ln & 15, g = ln >> 4;
      const int key = (base + n) * (kLatent * 2) + ((g ^ swz<LC>(n)) << 4);
      const int pos = kLatentBytes + (base + n) * (kRopeWidth * 2) + ((g ^ swz<8>(n)) << 4);
      // kAhead steps are on their way while one is used
      auto keys = [&](int k, v8s (&x)[NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          // chunk 4k + g: bits 0..3 xored with swz, the rest added
          const int at = k < KL ? (key ^ ((k & 3) << 6)) + (k >> 2) * 256 + t * 16 * (kLatent * 2)
                                : (pos ^ ((k - KL) << 6)) + t * 16 * (kRopeWidth * 2);
          x[t] = *(MXIDX_LDS const v8s*)(buf + at);
        }
      };
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (kMx && HG > 2) {
        // operand by operand, so that three of them do: two whole steps ahead spill a register of the query
        auto key_of = [&](int e) __attribute__((always_inline)) {
          const int k = e / NT, t = e % NT;
          return *(MXIDX_LDS const v8s*)(buf + (k < KL ? (key ^ ((k & 3) << 6)) + (k >> 2) * 256 + t * 16 * (kLatent * 2)
                                                       : (pos ^ ((k - KL) << 6)) + t * 16 * (kRopeWidth * 2)));
        };
        constexpr int kRing = 3;
        v8s x[kRing];
#pragma unroll
        for (int e = 0; e < kRing; ++e) x[e] = key_of(e);
#pragma unroll
        for (int e = 0; e < KS * NT; ++e) {
          __builtin_amdgcn_sched_barrier(0);
          s[e % NT] = mfma_bf16(x[e % kRing], q[e / NT], s[e % NT]);
          if (e + kRing < KS * NT) x[e % kRing] = key_of(e + kRing);
        }
      } else {
        v8s x[kAhead][NT];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) keys(k, x[k]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t = 0; t < NT; ++t) s[t] = mfma_bf16(x[k % kAhead][t], q[k], s[t]);
          if (k + kAhead < KS) keys(k + kAhead, x[k % kAhead]);
          if constexpr (!kMx) {
#pragma unroll
            for (int i = 0; i < Copy::kPieces; ++i)
              if (i * KS / Copy::kPieces == k)
                Copy::piece(i, cache, nxt, wave * kMine, rows, ln);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // s[t][i]: token base + 16t + 4g + i of this lane's head
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[t][i] *= scale2;
    if (mask != (kTile == 64 ? ~0ull : (1ull << (kTile % 64)) - 1)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t bits = (uint32_t)(mask >> (base + 16 * t + 4 * (fresh_lane() >> 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = (bits >> i) & 1 ? s[t][i] : neg_inf();
      }
    }
    float top = neg_inf();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
    top = max_groups(top);
    // the reference is raised only where weights would pass 2^kSlack: what was summed so
    // far is seldom rescaled
    const bool grow = m != neg_inf() && top > m + kSlack;
    const float m2 = grow || m == neg_inf() ? top : m;
    if (__any(grow)) {
      const float f = grow ? __builtin_amdgcn_exp2f(m - m2) : 1.f;
      l *= f;
#pragma unroll
      for (int v = 0; v < NV; ++v) o[v] *= f;
    }
    m = m2;
    const float ref = m == neg_inf() ? 0.f : m;      // no token yet: every weight 0
    uint32_t w[NT][2], rest[NT][2];                  // rest: what rounding left of the weights
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = __builtin_amdgcn_exp2f(s[t][i] - ref);
        l += p[i];
      }
      w[t][0] = pack2(p[0], p[1]);
      w[t][1] = pack2(p[2], p[3]);
      rest[t][0] = pack2(p[0] - low_half(w[t][0]), p[1] - high_half(w[t][0]));
      rest[t][1] = pack2(p[2] - low_half(w[t][1]), p[3] - high_half(w[t][1]));
    }
    // values: lane 4j + c of a 16-lane group reads tokens 4g + j, values 4c..4c+3, and
    // gets tokens 4g..4g+3 of value n
    const int vl = fresh_lane(), vn = vl & 15, vt = 4 * (vl >> 4) + (vn >> 2);
    const int val = (base + vt) * (kLatent * 2) + ((((vn >> 1) & 1) ^ swz<LC>(vt)) << 4) + 8 * (vn & 1);
    v4s y[kValuesAhead][NT];
    auto values = [&](int v, v4s (&x)[NT]) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MXIDX_LDS v4s*)(
            buf + (val ^ ((v & 7) << 5)) + (v >> 3) * 256 + t * 16 * (kLatent * 2)));
    };
    auto product = [&](const v4s (&z)[NT], const uint32_t (&by)[NT][2], v4f c) __attribute__((always_inline)) {
      if constexpr (NT == 1)
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
            z[0], __builtin_bit_cast(v4s, uint2{by[0][0], by[0][1]}), c, 0, 0, 0);
      else
        return mfma_bf16(__builtin_shufflevector(z[0], z[NT - 1], 0, 1, 2, 3, 4, 5, 6, 7),
                         __builtin_bit_cast(v8s, uint4{by[0][0], by[0][1], by[NT - 1][0], by[NT - 1][1]}), c);
    };
    const uint32_t there = (uint32_t)(next_mask >> (wave * kMine));
    if constexpr (kMx && kSpare) {
      mx.prepare(wave * kMine, (uint32_t)fresh_lane());
      mx.take(0, raw, 0, there);
    }
#pragma unroll
    for (int v = 0; v < kValuesAhead; ++v) values(v, y[v]);
    // parts of the output at a time: two where a wave is alone on its SIMD, so that no sum waits
    // (1024 rows of 2048 tokens, 64 heads: 363 us with one, 367 with two)
    constexpr int kStep = HG <= 2 ? 2 : 1;
#pragma unroll
    for (int v = 0; v < NV; v += kStep) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kStep; ++i) o[v + i] = product(y[(v + i) % kValuesAhead], w, o[v + i]);
#pragma unroll
      for (int i = 0; i < kStep; ++i) o[v + i] = product(y[(v + i) % kValuesAhead], rest, o[v + i]);
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        if (v + i + kValuesAhead < NV) values(v + i + kValuesAhead, y[(v + i) % kValuesAhead]);
      if constexpr (kMx) {
        // the next tile's codes on their way.  With registers to spare a dword at a time all along the
        // product, each read a step before it is written (1024 rows of 2048 tokens, 16 heads: 256 us, 270
        // with four at a time in its second half); else two at a time in its second half, written one after
        // the other, as their values take four registers each
        if constexpr (kSpare) {
          constexpr int kGap = NV / Mx::kDwords;
          static_assert(kGap % kStep == 0 && kGap > 0, "a step of its own for each");
          if (v % kGap == 0) {
            if (v / kGap + 1 < Mx::kDwords) mx.take(v / kGap + 1, raw, 0, there);
            mx.write(v / kGap, nxt);
          }
        } else {
          constexpr int kGap = NV / Mx::kDwords;       // half a product for twice as many
          static_assert(kGap > kStep && kGap % (2 * kStep) == 0, "steps of their own");
          const int u = 2 * ((v - NV / 2) / kGap);
          if (v >= NV / 2 && (v - NV / 2) % kGap == 0) {
            const uint32_t ln = (uint32_t)fresh_lane();
            if (u == 0) mx.prepare(wave * kMine, ln);
            mx.take(u, raw, ln, there);
            mx.take(u + 1, raw, ln, there);
          }
          if (v >= NV / 2 && (v - NV / 2) % kGap == kGap / 2) {
            mx.write(u, nxt);
            __builtin_amdgcn_sched_barrier(0);
            mx.write(u + 1, nxt);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // the pipeline: the tile computed, the next one's rows on their way to LDS, the one
  // behind it looking up its pages and the one behind that its list entries
  if (t0 < t1) {
    // a place past the list for lanes without a token
    auto place = [&](int t) {
      const int ln = fresh_lane();
      return kTile == kWave || ln < kTile ? t * kTile + ln : 0x7fffffff;
    };
    auto entry = [&](int t) { return list_entry(a, r, place(min(t, t1 - 1))); };
    const int e0 = entry(t0), e1 = entry(t0 + 1);
    int far = entry(t0 + 2);
    const int now = token_of(a, row, e0, place(t0));
    const int now_page = token_page(a, row, now);
    int next = token_of(a, row, e1, place(t0 + 1));
    int page = token_page(a, row, next);
    uint64_t mask;
    auto copy_all = [&](const Source& src, MXIDX_LDS uint8_t* tile, int rows) __attribute__((always_inline)) {
      const int ln = fresh_lane();
#pragma unroll
      for (int i = 0; i < Copy::kPieces; ++i) Copy::piece(i, src, tile, wave * kMine, rows, ln);
    };
    // the query's rows, as if they were a tile's, to LDS: as many heads as a tile has tokens to
    // tile1 behind the list's and pages' loads, and with 32-token tiles the others to tile0
    // before the tile
    constexpr int kQTiles = (kHeads + kTile - 1) / kTile;
#pragma unroll
    for (int i = 0; i < kQTiles; ++i) {
      const int h = i * kTile + fresh_lane(), head = group * kHeads + h;
      const uint32_t at = kSmall ? (uint32_t)head * (uint32_t)(a.q_head_stride * 2) : (uint32_t)head;
      copy_all(Source{static_cast<const char*>(a.q) + r * a.q_row_stride * 2, parts.q_bytes, a.q_head_stride * 2},
               (MXIDX_LDS uint8_t*)(i == 0 ? tile1 : tile0), h < kHeads && head < a.H ? (int)at : kNoRow);
    }
    const int first_rows = rows_of(now, now_page, mask);
    auto copy_first = [&]() __attribute__((always_inline)) {
      if constexpr (kMx) {
        const int ln = fresh_lane();
        mx.load(cache, raw, wave * kMine, first_rows, ln);
#pragma unroll
        for (int i = 0; i < Mx::kPosPieces; ++i)
          Mx::position(i, cache, (MXIDX_LDS uint8_t*)tile0, wave * kMine, first_rows, ln);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        mx.prepare(wave * kMine, ln);
#pragma unroll
        for (int u = 0; u < Mx::kDwords; ++u) {
          mx.take(u, raw, ln, (uint32_t)(mask >> (wave * kMine)));
          mx.write(u, (MXIDX_LDS uint8_t*)tile0);
        }
      } else {
        copy_all(cache, (MXIDX_LDS uint8_t*)tile0, first_rows);
      }
    };
    if (kQTiles == 1) copy_first();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    {
      const int ln = fresh_lane(), n = ln & 15, g = ln >> 4, h = (hg * 16 + n) % kTile;
      const int key = h * (kLatent * 2) + ((g ^ swz<LC>(n)) << 4);
      const int pos = kLatentBytes + h * (kRopeWidth * 2) + ((g ^ swz<8>(n)) << 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int at = k < KL ? (key ^ ((k & 3) << 6)) + (k >> 2) * 256 : pos ^ ((k - KL) << 6);
        q[k] = kQTiles > 1 && hg >= kTile / 16 ? *(MXIDX_LDS const v8s*)((MXIDX_LDS uint8_t*)tile0 + at)
                                               : *(MXIDX_LDS const v8s*)((MXIDX_LDS uint8_t*)tile1 + at);
      }
    }
    if (kQTiles > 1) {
      __syncthreads();
      copy_first();
    }
    // kMx: the codes of the tile behind the next one computed, on their way while that is
    int rows = kNoRow;
    uint64_t next_mask = 0;
    auto load_codes = [&](int t) __attribute__((always_inline)) {
      rows = rows_of(t < t1 ? next : -1, page, next_mask);
      // in this place: the count of the step's wait relies on it
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (t < t1) mx.load(cache, raw, wave * kMine, rows, fresh_lane());
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
    };
    if constexpr (kMx) load_codes(t0 + 1);
    // tile t from `cur`, tile t + 1 on its way to `nxt` (behind the last one: zeros)
    auto step = [&](int t, MXIDX_LDS uint8_t* cur, MXIDX_LDS uint8_t* nxt) __attribute__((always_inline)) {
      if constexpr (kMx) {
        // but for the next tile's codes and scales, whose loads are the youngest (a barrier of the
        // language would wait for them too)
        if (t + 1 < t1)
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(Mx::kYoungest) : "memory");
        else
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
      }
      if constexpr (!kMx) rows = rows_of(t + 1 < t1 ? next : -1, page, next_mask);
      next = token_of(a, row, far, place(t + 2));
      page = token_page(a, row, next);
      far = entry(t + 3);
      seen |= mask != 0;
      compute(cur, mask, nxt, rows, next_mask);
      mask = next_mask;
      if constexpr (kMx) load_codes(t + 2);
    };
    for (int t = t0; t < t1; t += 2) {
      step(t, (MXIDX_LDS uint8_t*)tile0, (MXIDX_LDS uint8_t*)tile1);
      if (t + 1 < t1) step(t + 1, (MXIDX_LDS uint8_t*)tile1, (MXIDX_LDS uint8_t*)tile0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last copies write LDS no more
  }

  // the waves' maxima and sums, and with them each one's factor
  const int ln = threadIdx.x & (kWave - 1), n = ln & 15, g = ln >> 4;
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if constexpr (kMx) __syncthreads();                  // the codes before have been read
  if (g == 0) stats[th][hg * 16 + n] = make_float2(m, l);
  __syncthreads();                                     // and the last tile's reads are done
  float f = 1.f;
  if constexpr (TH > 1) {
    float top = m, mine = m;
#pragma unroll
    for (int t = 0; t < TH; ++t) top = fmaxf(top, stats[t][hg * 16 + n].x);
    const float ref = top == neg_inf() ? 0.f : top;
    f = __builtin_amdgcn_exp2f(mine - ref);
    m = top;
    l = 0.f;
#pragma unroll
    for (int t = 0; t < TH; ++t) {
      const float2 other = stats[t][hg * 16 + n];
      l += __builtin_amdgcn_exp2f(other.x - ref) * other.y;
    }
  }
  const bool whole = parts.splits == 1;
  const int head = group * kHeads + hg * 16 + n;
  const int64_t part = (r * parts.splits + split) * parts.heads + group * kHeads;
  if (th == 0 && g == 0) {
    if (!whole)
      *reinterpret_cast<float2*>(parts.ml + 2 * (part + hg * 16 + n)) = make_float2(m, l);
    else if (a.lse && head < a.H)
      a.lse[r * a.H + head] = l == 0.f ? neg_inf() : m * 0.6931471805599453f + logf(l);
  }
  if (!whole && !seen) return;                         // uniform: the join does not read its sums
  if (whole) f *= l == 0.f ? 0.f : 1.f / l;

  // o[v][i] is value 16v + 4g + i of this lane's head: through LDS (16-byte chunk c of
  // head n at place c ^ n) into whole rows, the token parts added on the way, kValues
  // values at a time; each token part begins with a share of its own
  constexpr int kValues = HG <= 2 * (kTileBytes / (kLatent * 64)) ? kLatent : kLatent / 2;
  constexpr int CP = kValues / 4;                      // chunks of a row
  constexpr int kRegion = 16 * kValues * 4, kRegions0 = kTileBytes / kRegion;
  constexpr int NQ = kValues / 16 / TH;                // 16-value parts of a share
  static_assert(HG <= 2 * kRegions0, "the sums fit the tiles");
  auto region = [&](int i) { return i < kRegions0 ? tile0 + i * kRegion : tile1 + (i - kRegions0) * kRegion; };
#pragma unroll
  for (int v0 = 0; v0 < kLatent; v0 += kValues) {
    if (v0 > 0) __syncthreads();                       // the rows before have been read
    uint8_t* dst = region(hg) + n * (kValues * 4);
#pragma unroll
    for (int t = 0; t < TH; ++t) {
#pragma unroll
      for (int share = 0; share < TH; ++share) {
        if ((th + t) % TH != share) continue;          // uniform over the wave
        v4f x[NQ];
#pragma unroll
        for (int v = 0; v < NQ; ++v) {
          x[v] = o[v0 / 16 + share * NQ + v] * f;
          if (t > 0) x[v] += *reinterpret_cast<const v4f*>(dst + (((4 * (share * NQ + v) + g) ^ n) << 4));
        }
#pragma unroll
        for (int v = 0; v < NQ; ++v)
          *reinterpret_cast<v4f*>(dst + (((4 * (share * NQ + v) + g) ^ n) << 4)) = x[v];
      }
      __syncthreads();
    }
#pragma unroll 8
    for (int i = threadIdx.x; i < kHeads * CP; i += kWaves * kWave) {
      const int h = i / CP, c = i % CP;
      const v4f x = *reinterpret_cast<const v4f*>(region(h / 16) + (h % 16) * (kValues * 4) + ((c ^ (h % 16)) << 4));
      if (!whole) {
        *reinterpret_cast<v4f*>(parts.o + (part + h) * kLatent + v0 + 4 * c) = x;
      } else if (group * kHeads + h < a.H) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * a.out_row_stride +
                                  (int64_t)(group * kHeads + h) * a.out_head_stride + v0 + 4 * c) =
            make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
      }
    }
  }
}

// The splits' sums of one (row, head) by kGroups * kLatent / 4 lanes: 4 values each, a group of
// lanes takes every kGroups-th split, the loads of kBatch splits together (past the last
// one, its sums again), and with more groups than one LDS joins those, one (row, head) a workgroup.
template <int kLatent, int kBatch, int kGroups>
__global__ __launch_bounds__(kGroups == 1 ? 256 : kGroups * kLatent / 4) void attn_join_kernel(AttnArgs a,
                                                                                            Parts parts) {
  constexpr int W = kLatent / 4, kThreads = kGroups == 1 ? 256 : kGroups * W;
  __shared__ v4f sums[kGroups > 1 ? kGroups - 1 : 1][W];
  __shared__ float2 tops[kGroups > 1 ? kGroups - 1 : 1][W];
  const int64_t at = kGroups == 1 ? ((int64_t)blockIdx.x * kThreads + threadIdx.x) / W : (int64_t)blockIdx.x;
  const int i = threadIdx.x % W, group = kGroups == 1 ? 0 : threadIdx.x / W;
  const int64_t r = (uint32_t)at / (uint32_t)a.H;      // rows * H < 2^31
  const int head = (int)(at - r * a.H);
  Row row;
  if (r >= a.rows || !row_of(a, r, row)) return;       // with groups uniform over the workgroup
  const int64_t first = r * parts.splits * parts.heads + head;
  v4f o = {0.f, 0.f, 0.f, 0.f};
  float top = neg_inf(), l = 0.f;
  // what another has summed: o * 2^-top, l * 2^-top
  auto add = [&](float m, float ml, const v4f& x) __attribute__((always_inline)) {
    if (ml == 0.f) return;                             // nothing seen: no sums written
    const float f = __builtin_amdgcn_exp2f(m - (top == neg_inf() ? 0.f : top));
    l += f * ml;
    o += f * x;
  };
  auto raise = [&](float m) __attribute__((always_inline)) {
    const float old = __builtin_amdgcn_exp2f(top - (m == neg_inf() ? 0.f : m));
    o *= old;
    l *= old;
    top = m;
  };
  for (int s0 = group; s0 < parts.splits; s0 += kBatch * kGroups) {
    float2 ml[kBatch];
    v4f x[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int64_t p = first + (int64_t)min(s0 + s * kGroups, parts.splits - 1) * parts.heads;
      ml[s] = *reinterpret_cast<const float2*>(parts.ml + 2 * p);
      x[s] = *reinterpret_cast<const v4f*>(parts.o + p * kLatent + 4 * i);
    }
    float m = top;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) m = fmaxf(m, ml[s].x);
    raise(m);
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s * kGroups < parts.splits) add(ml[s].x, ml[s].y, x[s]);
  }
  if constexpr (kGroups > 1) {
    if (group > 0) {
      sums[group - 1][i] = o;
      tops[group - 1][i] = make_float2(top, l);
    }
    __syncthreads();
    if (group > 0) return;
    float m = top;
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g) m = fmaxf(m, tops[g][i].x);
    raise(m);
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g) add(tops[g][i].x, tops[g][i].y, sums[g][i]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * a.out_row_stride +
                            (int64_t)head * a.out_head_stride + 4 * i) =
      make_uint2(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv));
  if (a.lse && i == 0)
    a.lse[r * a.H + head] = l == 0.f ? neg_inf() : top * 0.6931471805599453f + logf(l);
}

struct Plan {
  int group_heads;        // heads of a workgroup
  int tile;               // tokens at a time
  int heads;              // H rounded up to whole groups
  int splits;
};

// Few rows are split over the tokens, up to one workgroup for each CU (two of latent 128, whose
// tiles leave the LDS room: 32 windows of 8192, 128 heads: 45.8 us, 47.6 with one).  A split
// costs its share of the workspace's traffic (2 KB a head, written and read), so it takes 4
// tiles or more (16 rows of 2048 tokens, 32 heads: 22.0 us with 8 splits, 23.0 with 16), or
// 2 where even 64 workgroups do not come together (one row of 64 heads: 15.7 us with 16 splits
// of 32 heads, 17.7 with 8); one row of 131072 tokens, 64 heads, latent 128: 29 us with 128
// splits, 42 with 64.
// 64 heads a workgroup read the rows fewest times (16 x 2 rows of 6600 tokens, 128
// heads: 101 us with 64, 139 with 32; 64 rows of 2048 tokens, 64 heads: 54 and 56); 32
// heads spread a call over twice the CUs that would not fill them otherwise (one row:
// 15.7 us, 17.9 with 64) or fill them with half the partial sums (32 rows of 2048 tokens,
// 64 heads: 32 us with 4 splits, 35 with 64 heads and 8; 4 rows of 16384: 32 and 34).
// Many rows: two workgroups of four waves a CU, 32 tokens at a time, whose phases do not
// fall together (1024 rows of 2048 tokens, 64 heads: 377 us, 395 with one of
// eight waves); with 200 rows, which do not fill both places, 126 us and 114.
// Groups of 16 and 32 heads keep one form for few rows and many (1024 rows of 2048 tokens: 230 us
// with 16 heads, 277 with 32, 379 with 64).
int64_t split_places(int latent) { return latent <= 128 ? 2 * kCus : kCus; }

// Over the MXFP4 cache (mx) windows of up to 5, 4 and 3 tiles of latent 128, 256 and 512 are not split:
// the second launch costs as much as the tiles that it saves (one row of 8 heads, 129 tokens, in a
// graph and called one by one: 6.9 / 9.3 us, 8.0 / 12.1 split, latent 128; 8.6 / 9.4 and 9.8 / 11.9,
// 256; 12.0 / 12.0 and 12.4 / 12.8, 512; of 385 tokens, latent 256, 13.4 / 13.4 and 10.2 / 11.9).
Plan plan_of(int64_t rows, int H, int latent, int64_t entries, bool mx) {
  Plan p;
  const int64_t tiles = (entries + 63) / 64, quarter = std::min<int64_t>((tiles + 3) / 4, kMaxSplits);
  const int64_t places = split_places(latent);
  p.group_heads = H <= 16 ? 16 : H <= 32 || rows * ((H + 31) / 32) * quarter <= 2 * kCus ? 32 : 64;
  p.heads = (H + p.group_heads - 1) / p.group_heads * p.group_heads;
  const int64_t units = rows * (p.heads / p.group_heads);
  p.tile = p.group_heads == 64 && units >= 2 * kCus ? 32 : 64;
  const int64_t shares = units * quarter <= 64 ? std::min<int64_t>((tiles + 1) / 2, kMaxSplits) : quarter;
  p.splits = (int)std::max<int64_t>(1, std::min(places / std::max<int64_t>(units, 1), shares));
  if (mx && tiles <= (latent == 128 ? 5 : latent == 256 ? 4 : 3)) p.splits = 1;
  return p;
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Of the partial sums of so many (row, split, head).
int64_t ml_bytes(int64_t parts) { return align256(parts * 8); }
int64_t part_bytes(int64_t parts, int latent) { return ml_bytes(parts) + parts * latent * 4; }

template <int kLatent, bool kMx>
hipError_t launch(const AttnArgs& a, void* workspace, hipStream_t stream) {
  const Plan p = plan_of(a.rows, a.H, kLatent, a.indices ? a.k : a.max_tokens, kMx);
  const int64_t cache_bytes = a.num_pages * (kMx ? mx_page_bytes(kLatent) : kPage * (kLatent + kRopeWidth) * 2);
  const int64_t q_bytes = ((a.H - 1) * a.q_head_stride + kLatent + kRopeWidth) * 2;
  const bool small = cache_bytes <= kReach && q_bytes <= kReach;
  Parts parts{nullptr, nullptr, p.splits, p.heads, (int)a.num_pages,
              small ? (uint32_t)cache_bytes : 0, small ? (uint32_t)q_bytes : 0};
  if (p.splits > 1) {
    parts.ml = static_cast<float*>(workspace);
    parts.o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(a.rows * p.splits * p.heads));
  }
  const dim3 grid((uint32_t)(a.rows * (p.heads / p.group_heads) * p.splits));
#define MXIDX_ATTN(heads_, tile_, hg, th)                                                     \
  case heads_ * 64 + tile_:                                                                   \
    if (small)                                                                               \
      hipLaunchKernelGGL((attn_kernel<kLatent, tile_, hg, th, true, kMx>), grid,             \
                         dim3(hg * th * kWave), 0, stream, a, parts);                        \
    else                                                                                     \
      hipLaunchKernelGGL((attn_kernel<kLatent, tile_, hg, th, false, kMx>), grid,            \
                         dim3(hg * th * kWave), 0, stream, a, parts);                        \
    break;
  switch (p.group_heads * 64 + p.tile) {
    MXIDX_ATTN(16, 64, 1, 4)
    MXIDX_ATTN(32, 64, 2, 2)
    MXIDX_ATTN(64, 64, 4, 2)
    MXIDX_ATTN(64, 32, 4, 1)
    default: return hipErrorInvalidValue;
  }
#undef MXIDX_ATTN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  constexpr int W = kLatent / 4;
  const int64_t threads = a.rows * a.H * W;
  const dim3 join((uint32_t)((threads + 255) / 256));
  // no loads beyond the splits that there are, as far as a power of two goes (2 splits of 64
  // rows, 128 heads: 10.2 us, 13.4 with eight loads; 4 of 32 rows: 8.8 and 9.9), and more lanes
  // where few rows have many splits (one row of 32768 tokens, 64 heads, 64 splits: 27.6 us
  // with four groups, 33.5 with one; 16 splits: 15.1 and 15.4)
  if (p.splits <= 2)
    hipLaunchKernelGGL((attn_join_kernel<kLatent, 2, 1>), join, dim3(256), 0, stream, a, parts);
  else if (p.splits <= 4)
    hipLaunchKernelGGL((attn_join_kernel<kLatent, 4, 1>), join, dim3(256), 0, stream, a, parts);
  else if (p.splits <= 8)
    hipLaunchKernelGGL((attn_join_kernel<kLatent, 8, 1>), join, dim3(256), 0, stream, a, parts);
  else
    hipLaunchKernelGGL((attn_join_kernel<kLatent, 8, 4>), dim3((uint32_t)(a.rows * a.H)), dim3(4 * W), 0, stream,
                       a, parts);
  return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t rows, int H, int latent, int64_t entries, bool mx) {
  const Plan p = plan_of(rows, H, latent, entries, mx);
  return p.splits == 1 ? 0 : part_bytes(rows * p.splits * p.heads, latent);
}

// Split rows come to at most `places` workgroups of the largest group that so few heads take, and
// to so many splits of the heads rounded up to it.
int64_t attn_workspace_max_bytes(int64_t rows, int H, int latent, int64_t entries) {
  const int64_t group = H <= 16 ? 16 : H <= 32 ? 32 : 64, heads = (H + group - 1) / group * group;
  const int64_t tiles = (entries + 63) / 64, splits = std::min<int64_t>((tiles + 1) / 2, kMaxSplits);
  return splits <= 1 ? 0 : part_bytes(std::min(split_places(latent) * group, rows * heads * splits), latent);
}

hipError_t launch_attn_paged(const AttnArgs& a, int latent, bool mx, void* workspace, hipStream_t stream) {
  switch (latent) {
    case 128: return mx ? launch<128, true>(a, workspace, stream) : launch<128, false>(a, workspace, stream);
    case 256: return mx ? launch<256, true>(a, workspace, stream) : launch<256, false>(a, workspace, stream);
    default: return mx ? launch<512, true>(a, workspace, stream) : launch<512, false>(a, workspace, stream);
  }
}

}  // namespace mxidx
