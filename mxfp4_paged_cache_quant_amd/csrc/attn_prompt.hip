// Attention of packed prompts over contiguous keys and values (idx_attn_prompt): for query row i of
// a request of `len` tokens, `new` of them rows of this call, and head h of key / value head h / G,
//   s_j = scale * q[i,h] . k_j,  out = sum_j exp(s_j - m) v_j / l,  l = sum_j exp(s_j - m),
//   lse = m + log l,  m = max_j s_j
// over the request's tokens j (causal: those up to position len - new + i).
//
// One pass over the tokens with the running maximum and sum (in powers of two): a new maximum
// scales what was summed so far by 2^(m_old - m_new).
//
// Work mapping: a workgroup takes `slots` of one request, 32 a wave: a slot is a query row and one
// of the G heads that share a key / value head, so that rows of few tokens fill a wave with heads.
// It walks the request's tokens 64 (a tile) at a time, keys and values going straight to LDS (two
// tiles, the next one's copies under the current one's products).  Products run on the 32x32x16
// bf16 MFMA in the transposed form:
//   S^T = K Q^T   A = 32 tokens of the tile, B = the wave's 32 slots
//   O^T = V^T P^T A = 32 of the values over 16 tokens, B = the weights
// so a lane (and the one 32 lanes on) holds one slot throughout: the weights leave the first product
// in the registers where the second takes them (half h of the lanes: tokens 4h..4h+3 and
// 8+4h..8+4h+3 of 16), and the running maximum and sum are one register each.
//
// The weights go to the second product rounded to bf16 (2^-8), relative to the running maximum itself, so
// that a token that dominates a row weighs exactly 1; l and lse take them unrounded.  Where the roundings of
// many different weights average out the output's error is 1.06-1.10 times its own rounding's.
// Equal weights all round the same way: where one token has the maximum and thousands share a lower
// score, the output is off by up to 2^-8 of itself beside its own rounding, of 2^-8 too.
// Divided by the sum of the rounded weights it would not be (16 dot products with ones a tile more), but
// every instruction counts here: a prompt of 16384 tokens 1247 -> 1307 us, of 8192 tokens, heads of 128, 293 -> 303, heads of
// 64 170 -> 182, for errors of 1.05-1.09.  A second part of the weights, as the attention over the
// cache has it, would be half as many products again where the products are what bounds the kernel.
//
// What bounds it: with many rows the card's power.  A prompt of 16384 tokens, 16 heads of 192 / 128,
// takes 1.25-1.3 ms = 1,050-1,100 TFLOP/s at 1.4-1.7 GHz, where a large library product reaches
// 1,310-1,400 (inputs of zeros: 0.9 ms); of the SIMDs' cycles 60% are MFMAs, and no LDS access
// meets a bank conflict.  Smaller heads are bound by instruction issue: the softmax of a tile is the same
// work beside 32 MFMAs (128) or 16 (64) as beside 40 (192 / 128), so that 6.0 and 11.4 other vector
// instructions go with an MFMA, 4.5 there; MFMAs are busy 45% and 37% of the time at 1.9-2.0 GHz, and waves
// wait for an issue slot 40-43% of their cycles.  Steps: operands kept three and four steps ahead (1286 -> 1247 us; heads of
// 64, four prompts of 4000, 191 -> 169); two to four steps ahead, values read before the weights
// are there, and a wave priority for the products: all within 1%.  Scores a tile ahead of the weights in
// one wave (its registers are full): 298 and 303 us for a prompt of 8192 tokens, 16 heads of 128.  Eight
// waves a workgroup: 3% faster there, 40% slower for heads of 64, 2% for packed prompts of 1000.
// With few rows over many tokens it is HBM: 64 rows, 32 heads of 128 on 4, over 1000-8192 tokens each
// 120 us = 5.0 TB/s, where a large copy makes 4.7-4.9.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

constexpr int kTile = 64;                   // tokens at a time
constexpr int kWaveSlots = 32;
constexpr int kAhead = 3, kValuesAhead = 4;   // operand steps of the products on their way
constexpr int kMinShare = 4;                // tiles that a share of a split row walks at least

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
#define MXIDX_LDS __attribute__((address_space(3)))

__device__ __forceinline__ v16f mfma32(v8s a, v8s b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// The larger of a lane's value and that of the lane 32 on, and their sum.
__device__ __forceinline__ float max_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// LDS place of a 16-byte chunk: chunk c of token t's row at c ^ swz(t).  Keys are read a chunk of 32
// tokens at a time, values four chunks of eight tokens by transposing reads.
template <int C>                            // chunks of a row: 16 (256 bytes) or 8
__device__ __forceinline__ int key_swz(int t) { return C == 16 ? t & 15 : (t >> 1) & 7; }
template <int C>
__device__ __forceinline__ int value_swz(int t) { return C == 16 ? (t & 3) << 2 : ((t >> 1) & 1) << 2; }

// The inclusive sum over a wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
#define MXIDX_ADD(control, rows) x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, control, rows, 0xf, true)
  MXIDX_ADD(0x111, 0xf);                    // one, two, four and eight lanes up in rows of 16
  MXIDX_ADD(0x112, 0xf);
  MXIDX_ADD(0x114, 0xf);
  MXIDX_ADD(0x118, 0xf);
  MXIDX_ADD(0x142, 0xa);                    // the first and third row's sum to the second and fourth
  MXIDX_ADD(0x143, 0xc);                    // the lower half's to the upper
#undef MXIDX_ADD
  return x;
}

// How the rows are dealt out.  Slots are blocks of `heads` heads by `tok` rows (a tile); without shares each
// tile of a head block is one item, of a workgroup.  With them a head block has `items`, more than it
// has tiles, and the requests' tiles are cut into shares of about equal length, whatever the requests'
// lengths: each leaves for each of its slots unscaled sums and (m, l), which a second launch joins.
struct PromptParts {
  float* o;                // [head block, item, slot, kDv]
  float* ml;
  int tok, heads, blocks;  // rows of a tile; heads of a block, blocks of a key head's
  uint32_t tiles, items;   // of a head block: tiles at most, items
  bool shares;
};

__device__ __forceinline__ float wave_sum(float x) {
#define MXIDX_ADD(control, rows) \
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), control, rows, 0xf, true))
  MXIDX_ADD(0x111, 0xf);
  MXIDX_ADD(0x112, 0xf);
  MXIDX_ADD(0x114, 0xf);
  MXIDX_ADD(0x118, 0xf);
  MXIDX_ADD(0x142, 0xa);
  MXIDX_ADD(0x143, 0xc);
#undef MXIDX_ADD
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), kWave - 1));
}

// A request's tile of query rows, where its rows, keys and values begin, and its share or shares.
struct Found {
  int64_t row, key;        // the first query row and the first key of the request
  int n, len, pos0;        // its rows and its keys that there are, the position of its first row
  int tile;                // -1: no such tile
  int share, shares;
  uint32_t item, step;     // the tile's first item, and from one of its shares' to the next
};

// Item (kByItem) or tile `want` of all requests', a request's last rows, which see most, first.  Every
// wave looks for itself, 64 requests at a time.
template <bool kByItem>
__device__ Found find(const PromptArgs& a, const PromptParts& parts, uint32_t want) {
  const int ln = threadIdx.x & (kWave - 1);
  const uint32_t T = (uint32_t)a.T, tok = (uint32_t)parts.tok;   // T below 2^23: sums of 64 fit 32 bits
  uint32_t row0 = 0, tile0 = 0, item0 = 0;
  int64_t key0 = 0;
  int n, len, next_n, next_len;                        // the next 64 requests' on their way
  uint32_t row, row_end, there, tiles;
  auto fetch = [&](int b0) {
    const int b = b0 + ln;
    next_n = b < a.B ? a.query_lens[b] : 0;
    next_len = b < a.B ? a.seq_lens[b] : 0;
  };
  auto load = [&](int b0) {
    n = max(next_n, 0);
    len = max(next_len, 0);
    fetch(b0 + kWave);
    const uint32_t mine = min((uint32_t)n, T);
    row_end = wave_scan(mine) + row0;
    row = row_end - mine;
    there = row < T ? min(mine, T - row) : 0;
    tiles = (there + tok - 1) / tok;
  };
  auto key_tiles = [&]() { return (uint32_t)((min((int64_t)len, a.max_seq_len) + kTile - 1) / kTile); };
  auto last_of = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, kWave - 1); };
  uint32_t length = ~0u;                               // of a share
  if (parts.shares) {
    // sum(tiles * ceil(key tiles / length)) <= sum(tiles * key tiles) / length + sum(tiles) <= items; the
    // products' and sums' roundings, each of 2^-24, come to less than 2^-8
    float work = 0.f;
    uint32_t all = 0;
    fetch(0);
    for (int b0 = 0; b0 < a.B; b0 += kWave) {
      load(b0);
      work += wave_sum((float)tiles * (float)key_tiles());
      all += last_of(wave_scan(tiles));
      row0 = min(last_of(row_end), T);
    }
    const float each = work / (float)(parts.items - all) * (1.f + 0x1p-8f);
    length = max((uint32_t)kMinShare, (uint32_t)ceilf(fminf(each, 0x1p30f)));
    row0 = 0;
  }
  Found f;
  f.tile = -1;
  fetch(0);
  for (int b0 = 0; b0 < a.B; b0 += kWave) {
    load(b0);
    const uint32_t shares = parts.shares ? max((key_tiles() + length - 1) / length, 1u) : 1u, items = tiles * shares;
    const uint32_t tile_end = wave_scan(tiles) + tile0, item_end = wave_scan(items) + item0;
    // the keys' sum in two halves of 16 bits: 64 of each fit
    const uint32_t low = wave_scan((uint32_t)len & 0xffffu), high = wave_scan((uint32_t)len >> 16);
    const uint32_t end = kByItem ? item_end : tile_end, mine = kByItem ? items : tiles;
    const uint64_t hit = __ballot(want < end && want >= end - mine);
    if (hit) {
      const int from = __builtin_ctzll(hit);
      auto of = [&](uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, from); };
      f.row = of(row);
      f.len = (int)of((uint32_t)len);
      f.n = (int)of(there);
      f.pos0 = f.len - (int)of((uint32_t)n);
      const int64_t key = key0 + ((int64_t)high << 16) + low - len;
      f.key = (int64_t)((uint64_t)of((uint32_t)((uint64_t)key >> 32)) << 32 | of((uint32_t)key));
      f.len = (int)min(min((int64_t)f.len, a.max_seq_len), max(a.S - f.key, (int64_t)0));
      f.shares = (int)of(shares);
      // a request's items: the tiles' first shares, their second ones ..., so that neighbours read the same keys
      f.step = of(tiles);
      const uint32_t in = want - of(end - mine), share = in / f.step, turn = in - share * f.step;   // tiles from the last
      f.share = (int)share;
      f.item = of(item_end - items) + turn;
      f.tile = (int)(f.step - 1 - turn);
      return f;
    }
    row0 = min(last_of(row_end), T);
    tile0 = last_of(tile_end);
    item0 = last_of(item_end);
    key0 += ((int64_t)last_of(high) << 16) + last_of(low);
  }
  return f;
}

// C chunks of each of 64 rows to LDS, kWaves waves sharing them: piece i of kPieces of a wave.
template <int C, int kWaves>
struct RowCopy {
  static constexpr int kPer = kWave / C, kPieces = kTile / kPer / kWaves;   // rows an instruction
  static_assert(kPieces * kPer * kWaves == kTile, "whole instructions");
  template <bool kKeys>
  static __device__ __forceinline__ void piece(int i, __amdgpu_buffer_rsrc_t rs, MXIDX_LDS uint8_t* dst,
                                               uint32_t stride, uint32_t offset, int wave, int ln) {
    const int t0 = (i * kWaves + wave) * kPer, t = t0 + ln / C;
    const int c = (ln % C) ^ (kKeys ? key_swz<C>(t) : value_swz<C>(t));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (MXIDX_LDS void*)(dst + t0 * C * 16), 16,
                                             (int)((uint32_t)t * stride + offset + (uint32_t)c * 16u), 0, 0, 0);
  }
};

template <int kDk, int kDv, int kWaves>
__global__ __launch_bounds__(kWaves * kWave, kWaves == 1 ? 1 : 2) void prompt_kernel(PromptArgs a, PromptParts parts) {
  constexpr int kA = kDk >= 128 ? 128 : 0, kB = kDk - kA;       // a key's 256-byte and 128-byte parts
  static_assert(kB == 0 || kB == 64, "key parts");
  constexpr int KS = kDk / 16, KA = kA / 16;                    // contraction steps, of the first part
  constexpr int NV = kDv / 32, VC = kDv / 8;                    // 32-value parts, chunks of a value row
  constexpr int kKeyA = kTile * kA * 2, kKeyB = kTile * kB * 2, kValue = kTile * kDv * 2;
  constexpr int kBytes = kKeyA + kKeyB + kValue;
  __shared__ __attribute__((aligned(1024))) uint8_t tile0[kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t tile1[kBytes];

  // each XCD takes a run of neighbouring numbers: the shares and tiles of one head, which read the
  // same keys and values
  const uint32_t xcd = blockIdx.x % 8, turn = blockIdx.x / 8;
  // (of four where there are shares: fewer than the items may be taken, and none of the XCDs gets the rest)
  const uint32_t number = parts.shares ? (turn / 4 * 8 + xcd) * 4 + turn % 4
                                       : xcd * (gridDim.x / 8) + min(xcd, gridDim.x % 8) + turn;
  const uint32_t hb = number / parts.items;
  if (hb >= (uint32_t)a.Hk * parts.blocks) return;     // the grid is whole runs
  const int kv_head = (int)(hb / (uint32_t)parts.blocks), block = (int)(hb - kv_head * (uint32_t)parts.blocks);
  const Found f = find<true>(a, parts, number - hb * parts.items);
  if (f.tile < 0) return;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), ln = threadIdx.x & (kWave - 1);
  const int half = ln >> 5, n = ln & 31;
  const int G = a.Hq / a.Hk, h0 = block * parts.heads, heads = min(parts.heads, G - h0);
  // this lane's slot: past the last row or head a live one's, not written
  const int slot = wave * kWaveSlots + n;
  const int row_in = slot / parts.heads, head_in = slot - row_in * parts.heads;
  const int i0 = f.tile * parts.tok, last = min(i0 + parts.tok, f.n) - 1;
  const int i = min(i0 + row_in, last);
  const bool live = i0 + row_in <= last && head_in < heads;
  const int64_t row = f.row + i;
  const int head = kv_head * G + h0 + min(head_in, heads - 1);
  auto limit = [&](int at) { return a.causal ? max(min(f.pos0 + at + 1, f.len), 0) : f.len; };   // visible: below it
  const int lim = limit(i);
  const int wave_lo = __builtin_amdgcn_readfirstlane(limit(min(i0 + wave * kWaveSlots / parts.heads, last)));
  const int wave_hi = __builtin_amdgcn_readfirstlane(limit(min(i0 + (wave * kWaveSlots + kWaveSlots - 1) / parts.heads, last)));
  const int end = __builtin_amdgcn_readfirstlane(limit(last));
  const int tiles = (end + kTile - 1) / kTile, each = tiles / f.shares, more = tiles - each * f.shares;
  const int t0 = f.share * each + min(f.share, more), t1 = t0 + each + (f.share < more ? 1 : 0);

  v8s q[KS];                                           // step s: values 16s + 8 half .. +7
  {
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + row * a.q_row_stride + head * a.q_head_stride + 8 * half;
#pragma unroll
    for (int k = 0; k < KS; ++k) q[k] = *reinterpret_cast<const v8s*>(src + 16 * k);
  }
  // scores in powers of two; a negative scale by the query's sign, so that a larger product is a larger score
  const float scale2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
  if (a.scale < 0.f) {
#pragma unroll
    for (int k = 0; k < KS; ++k) q[k] ^= (short)0x8000;
  }

  v16f o[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[v][j] = 0.f;
  float m = neg_inf(), l = 0.f;                        // l: this lane's tokens only

  const char* kbase = static_cast<const char*>(a.k) + (f.key * a.k_row_stride + kv_head * a.k_head_stride) * 2;
  const char* vbase = static_cast<const char*>(a.v) + (f.key * a.v_row_stride + kv_head * a.v_head_stride) * 2;
  const uint32_t kstride = (uint32_t)(a.k_row_stride * 2), vstride = (uint32_t)(a.v_row_stride * 2);
  auto copy = [&](int t, MXIDX_LDS uint8_t* tile) __attribute__((always_inline)) {
    // rows past the request's last are out of the descriptors' range and read as zeros
    const int left = min(f.len - t * kTile, kTile);
    const __amdgpu_buffer_rsrc_t kr =
        buffer_rsrc(kbase + (int64_t)t * kTile * kstride, (int)((uint32_t)(left - 1) * kstride + kDk * 2));
    const __amdgpu_buffer_rsrc_t vr =
        buffer_rsrc(vbase + (int64_t)t * kTile * vstride, (int)((uint32_t)(left - 1) * vstride + kDv * 2));
    if constexpr (kA > 0) {
#pragma unroll
      for (int i = 0; i < RowCopy<16, kWaves>::kPieces; ++i)
        RowCopy<16, kWaves>::template piece<true>(i, kr, tile, kstride, 0, wave, ln);
    }
    if constexpr (kB > 0) {
#pragma unroll
      for (int i = 0; i < RowCopy<8, kWaves>::kPieces; ++i)
        RowCopy<8, kWaves>::template piece<true>(i, kr, tile + kKeyA, kstride, kA * 2, wave, ln);
    }
#pragma unroll
    for (int i = 0; i < RowCopy<VC, kWaves>::kPieces; ++i)
      RowCopy<VC, kWaves>::template piece<false>(i, vr, tile + kKeyA + kKeyB, vstride, 0, wave, ln);
  };

  // Where a lane reads of a tile's values: lane 4j + c of a 16-lane group token 4 half + j, values 4c..4c+3 of its 16
  // (chunk 4v and on for part v: value_swz takes from a token what its steps of 8 leave as it is).  Opaque, as a
  // sum that the compiler spreads over steps of an address hides from it which tile a read is of, and it
  // then waits for the next one's copies before the reads.
  int value_at = (4 * half + ((ln & 15) >> 2)) * (kDv * 2) +
                 (((2 * ((ln >> 4) & 1) + ((ln & 3) >> 1)) ^ value_swz<VC>((ln & 15) >> 2)) << 4) + 8 * (ln & 1);
  asm("" : "+v"(value_at));

  auto compute = [&](int t, MXIDX_LDS const uint8_t* tile) __attribute__((always_inline)) {
    const int first = t * kTile;
    if (first >= wave_hi) return;                      // uniform: no slot sees the tile
    v16f s[2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[p][j] = 0.f;
    // kAhead steps' operands are on their way while one is used
    auto keys = [&](int k, v8s (&x)[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int tok = 32 * p + n;
        x[p] = *(MXIDX_LDS const v8s*)(tile + (k < KA ? tok * 256 + (((2 * k + half) ^ key_swz<16>(tok)) << 4)
                                                      : kKeyA + tok * 128 + (((2 * (k - KA) + half) ^ key_swz<8>(tok)) << 4)));
      }
    };
    {
      v8s x[kAhead][2];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) keys(k, x[k]);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 0; p < 2; ++p) s[p] = mfma32(x[k % kAhead][p], q[k], s[p]);
        if (k + kAhead < KS) keys(k + kAhead, x[k % kAhead]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // s[p][j]: token first + 32p + 8 (j / 4) + 4 half + j % 4
    if (first + kTile > wave_lo) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (first + 32 * p + 8 * (j / 4) + 4 * half + j % 4 >= lim) s[p][j] = neg_inf();
    }
    float top = neg_inf();
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[p][j]);
    top = max_halves(top) * scale2;
    const float m2 = fmaxf(m, top);
    if (__any(m2 > m)) {
      const float fac = m2 > m && m != neg_inf() ? __builtin_amdgcn_exp2f(m - m2) : 1.f;
      l *= fac;
#pragma unroll
      for (int v = 0; v < NV; ++v) o[v] *= fac;
    }
    m = m2;
    const float ref = m == neg_inf() ? 0.f : m;
    uint32_t w[4][4];                                  // 16-token step u: its weights, two a register
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float x = __builtin_amdgcn_exp2f(fmaf(s[p][j], scale2, -ref));
        const float y = __builtin_amdgcn_exp2f(fmaf(s[p][j + 1], scale2, -ref));
        l += x + y;
        w[2 * p + j / 8][(j % 8) / 2] = pack2(x, y);
      }
    auto values = [&](int i, v4s (&x)[2]) __attribute__((always_inline)) {
      const int u = i / NV, v = i % NV;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (MXIDX_LDS v4s*)(tile + ((value_at ^ (v << 6)) + kKeyA + kKeyB + (16 * u + 8 * e) * (kDv * 2))));
    };
    v4s y[kValuesAhead][2];
#pragma unroll
    for (int i = 0; i < kValuesAhead; ++i) values(i, y[i]);
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const int u = i / NV, v = i % NV;
      const v4s(&x)[2] = y[i % kValuesAhead];
      o[v] = mfma32(__builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7),
                    __builtin_bit_cast(v8s, uint4{w[u][0], w[u][1], w[u][2], w[u][3]}), o[v]);
      if (i + kValuesAhead < 4 * NV) values(i + kValuesAhead, y[i % kValuesAhead]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  if (t0 < t1) copy(t0, (MXIDX_LDS uint8_t*)tile0);
  auto step = [&](int t, MXIDX_LDS uint8_t* cur, MXIDX_LDS uint8_t* nxt) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t + 1 < t1) copy(t + 1, nxt);
    compute(t, cur);
  };
  for (int t = t0; t < t1; t += 2) {
    step(t, (MXIDX_LDS uint8_t*)tile0, (MXIDX_LDS uint8_t*)tile1);
    if (t + 1 < t1) step(t + 1, (MXIDX_LDS uint8_t*)tile1, (MXIDX_LDS uint8_t*)tile0);
  }

  l = sum_halves(l);
  if (!live) return;
  if (f.shares == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.lse && half == 0) a.lse[row * a.Hq + head] = l == 0.f ? neg_inf() : m * 0.6931471805599453f + logf(l);
    uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.out_row_stride + head * a.out_head_stride + 4 * half;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<uint2*>(dst + 32 * v + 2 * j) =
            make_uint2(pack2(o[v][j] * inv, o[v][j + 1] * inv), pack2(o[v][j + 2] * inv, o[v][j + 3] * inv));
  } else {
    const int64_t part = ((int64_t)hb * parts.items + f.item + f.share * f.step) * (kWaves * kWaveSlots) + slot;
    if (half == 0) *reinterpret_cast<float2*>(parts.ml + 2 * part) = make_float2(m, l);
    if (l == 0.f) return;                              // the join does not read its sums
    float* dst = parts.o + part * kDv + 4 * half;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(dst + 32 * v + 2 * j) = make_float4(o[v][j], o[v][j + 1], o[v][j + 2], o[v][j + 3]);
  }
}

// The shares' sums of a tile's slots: kDv / 4 lanes of 4 values take every kGroups-th share, kBatch loads
// together (past the last one, its sums again), and with more groups than one LDS joins those, in
// groups of one slot.
template <int kDv, int kSlots, int kGroups>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs a, PromptParts parts) {
  constexpr int W = kDv / 4, kAt = 256 / W / kGroups, kBatch = kGroups > 1 ? 8 : 4;     // slots of a workgroup
  __shared__ v4f sums[kGroups][kAt][W];
  __shared__ float2 stats[kGroups][kAt];
  const uint32_t per = kSlots / kAt, unit = blockIdx.x / per, hb = unit / parts.tiles;
  const Found f = find<false>(a, parts, unit - hb * parts.tiles);
  if (f.tile < 0 || f.shares == 1) return;
  const int i = threadIdx.x % W, which = threadIdx.x / W, group = which % kGroups, at = which / kGroups;
  const int slot = (int)(blockIdx.x - unit * per) * kAt + at;
  const int row_in = slot / parts.heads, head_in = slot - row_in * parts.heads;
  const int kv_head = (int)(hb / (uint32_t)parts.blocks), block = (int)(hb - kv_head * (uint32_t)parts.blocks);
  const int G = a.Hq / a.Hk, h0 = block * parts.heads, i0 = f.tile * parts.tok;
  const bool live = row_in < parts.tok && i0 + row_in < f.n && head_in < min(parts.heads, G - h0);
  const int64_t first = ((int64_t)hb * parts.items + f.item) * kSlots + slot;
  v4f o = {0.f, 0.f, 0.f, 0.f};
  float m = neg_inf(), l = 0.f;
  auto add = [&](float m2, float l2, const v4f& x) __attribute__((always_inline)) {
    if (l2 == 0.f) return;                             // nothing seen: no sums written
    const float top = fmaxf(m, m2), old = __builtin_amdgcn_exp2f(m - top), f2 = __builtin_amdgcn_exp2f(m2 - top);
    o = o * old + x * f2;
    l = l * old + l2 * f2;
    m = top;
  };
  if (live) {
    for (int s0 = group; s0 < f.shares; s0 += kBatch * kGroups) {
      float2 ml[kBatch];
      v4f x[kBatch];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const int64_t p = first + (int64_t)min(s0 + s * kGroups, f.shares - 1) * f.step * kSlots;
        ml[s] = *reinterpret_cast<const float2*>(parts.ml + 2 * p);
        x[s] = *reinterpret_cast<const v4f*>(parts.o + p * kDv + 4 * i);
      }
#pragma unroll
      for (int s = 0; s < kBatch; ++s)
        if (s0 + s * kGroups < f.shares) add(ml[s].x, ml[s].y, x[s]);
    }
  }
  if constexpr (kGroups > 1) {
    sums[group][at][i] = o;
    if (i == 0) stats[group][at] = make_float2(m, l);
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) add(stats[g][at].x, stats[g][at].y, sums[g][at][i]);
  }
  if (!live) return;
  const int64_t row = f.row + i0 + row_in;
  const int head = kv_head * G + h0 + head_in;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.out_row_stride + head * a.out_head_stride + 4 * i) =
      make_uint2(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv));
  if (a.lse && i == 0) a.lse[row * a.Hq + head] = l == 0.f ? neg_inf() : m * 0.6931471805599453f + logf(l);
}

struct Plan {
  int waves;               // of a workgroup, 32 slots each
  int heads, blocks;       // heads of a slot block, blocks of a key head's group
  int tok;                 // rows of a tile
  int64_t groups, tiles, items;   // head blocks; of one: tiles at most, items
};

// One wave a workgroup where a request's rows and a group's heads come to 32 slots, four else (64 requests,
// one row each, 32 heads on 4: 121 us, 152 with four waves; 16 requests of 5 rows, 40 slots: 57 and
// 61 with one).  Shares where the tiles alone leave workgroups' places free and windows are longer
// than one share: two workgroups of four waves a CU, whose LDS they fill (one: 129 us for 4 requests
// of 61 rows over 16000-65536 tokens, 122 so), or four of one wave, in two turns (64 requests of
// one row: 138 us with two a CU, 121 with four, 127 with eight).  A share walks 4 tiles or more
// (one row over 65536 tokens: 34 us, 44 with 8; three prompts of up to 129 tokens: 8 us, 14 with 2,
// for the second launch).
Plan plan_of(int64_t T, int Hq, int Hk, int B, int64_t max_seq_len) {
  Plan p;
  const int G = Hq / Hk;
  const int64_t seqs = std::min<int64_t>(B, T), each = (T + seqs - 1) / std::max<int64_t>(seqs, 1);   // rows of a request
  p.waves = each * G <= kWaveSlots ? 1 : 4;
  const int slots = p.waves * kWaveSlots;
  p.heads = std::min(G, slots);
  p.blocks = (G + p.heads - 1) / p.heads;
  p.tok = slots / p.heads;
  p.groups = (int64_t)Hk * p.blocks;
  p.tiles = T / p.tok + seqs;
  const int64_t room = (p.waves == 1 ? 1024 : 512) / p.groups;
  p.items = max_seq_len > kMinShare * kTile && room > p.tiles ? room : p.tiles;
  return p;
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

int64_t workgroups(const Plan& p) {
  return p.items == p.tiles ? p.groups * p.items : (p.groups * p.items + 31) / 32 * 32;
}

// Of the shares' statistics and sums, where there are shares.
int64_t ml_bytes(const Plan& p) { return align256(p.groups * p.items * p.waves * kWaveSlots * 8); }
int64_t part_bytes(const Plan& p, int dv) {
  return p.items == p.tiles ? 0 : ml_bytes(p) + p.groups * p.items * p.waves * kWaveSlots * dv * 4;
}

template <int kDk, int kDv>
hipError_t launch(const PromptArgs& a, void* workspace, hipStream_t stream) {
  const Plan p = plan_of(a.T, a.Hq, a.Hk, a.B, a.max_seq_len);
  PromptParts parts{nullptr, nullptr, p.tok, p.heads, p.blocks, (uint32_t)p.tiles, (uint32_t)p.items, p.items != p.tiles};
  if (parts.shares) {
    parts.ml = static_cast<float*>(workspace);
    parts.o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(p));
  }
  const dim3 grid((uint32_t)workgroups(p));
  if (p.waves == 1)
    hipLaunchKernelGGL((prompt_kernel<kDk, kDv, 1>), grid, dim3(kWave), 0, stream, a, parts);
  else
    hipLaunchKernelGGL((prompt_kernel<kDk, kDv, 4>), grid, dim3(4 * kWave), 0, stream, a, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !parts.shares) return e;
  // eight groups of lanes a slot where a tile may have many shares, up to 1024 of them (one row over
  // 65536 tokens: 25.2 us, 26.9 with batches of four), else a slot to each (4 requests of 61 rows: 113, 122)
  const bool many = p.items >= 24 * p.tiles;
  const int slots = p.waves * kWaveSlots, at = 256 / (kDv / 4) / (many ? 8 : 1);
  const dim3 join((uint32_t)(p.groups * p.tiles * (slots / at)));
#define MXIDX_JOIN(slots_, groups_) \
  hipLaunchKernelGGL((prompt_join_kernel<kDv, slots_, groups_>), join, dim3(256), 0, stream, a, parts)
  if (p.waves == 1) {
    if (many) MXIDX_JOIN(32, 8); else MXIDX_JOIN(32, 1);
  } else {
    if (many) MXIDX_JOIN(128, 8); else MXIDX_JOIN(128, 1);
  }
#undef MXIDX_JOIN
  return hipGetLastError();
}

}  // namespace

int64_t prompt_workspace_bytes(int64_t T, int Hq, int Hk, int dv, int B, int64_t max_seq_len) {
  return T == 0 || B == 0 ? 0 : part_bytes(plan_of(T, Hq, Hk, B, max_seq_len), dv);
}

int64_t prompt_lanes(int64_t T, int Hq, int Hk, int B, int64_t max_seq_len) {
  const Plan p = plan_of(T, Hq, Hk, B, max_seq_len);
  return workgroups(p) * p.waves * kWave;
}

hipError_t launch_attn_prompt(const PromptArgs& a, int dk, int dv, void* workspace, hipStream_t stream) {
  if (dk == 64 && dv == 64) return launch<64, 64>(a, workspace, stream);
  if (dk == 128 && dv == 128) return launch<128, 128>(a, workspace, stream);
  return launch<192, 128>(a, workspace, stream);
}

}  // namespace mxidx
