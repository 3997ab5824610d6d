// Attention over the paged latent cache (idx_attn_paged): for each query row r and
// head h, with row_j the cached row of visible token j and n the latent size,
//   s_j = scale * sum_i q[r,h,i] * row_j[i]  (n + 64 values),
//   out[r,h,:] = sum_j exp(s_j - m) * row_j[:n] / l,  l = sum_j exp(s_j - m),
//   lse[r,h] = m + log l,  m = max_j s_j.
//
// One pass over the tokens with the running maximum and sum (in powers of two): a
// new maximum scales what was summed so far by 2^(m_old - m_new).
//
// Work mapping: one workgroup takes HG * 16 heads of one query row over one share of
// the row's tokens, 64 tokens (a tile) at a time.  A wave holds 16 heads: their query
// in registers and their output sums, HG waves the heads and TH waves the tile's
// token parts.  All products run on the 16x16x32 bf16 MFMA in the transposed form:
//   S^T = K Q^T   A = 16 tokens of the tile, B = the wave's 16 heads
//   O^T = V^T P^T A = 16 of the n values over 32 tokens, B = the weights
// so a lane holds one head throughout: the weights leave the first product in the
// registers where the second takes them (lane group g: tokens 4g..4g+3 of two 16-token
// parts), and the running maximum and sum are one register each.
//
// A row serves as key and, in its first n values, as value, so each cached row is
// read once into LDS (two tiles, the next one's loads in flight behind the current
// one's products).  The copies go straight from the cache rows to LDS in 16-byte
// chunks; chunk c of token t lands at place c ^ swz(t) of the row, which spreads both
// the keys' reads (16 tokens, one chunk) and the values' transposing reads (16 tokens,
// two neighbouring chunks) over all banks.
//
// Places of a tile that hold no visible token read a visible token's row instead and
// get weight 0, so nothing that a masked place holds reaches a sum; a tile with no
// visible token is skipped.
//
// The weights are rounded to bf16 for the second product (relative error 2^-8 at most,
// as the cached values' own); l and lse take them unrounded.
//
// Few rows: the tokens are split over workgroups, each leaving its unscaled sums with
// m and l in the workspace, and a second launch joins them.
#include "common.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

constexpr int kRopeWidth = 64;
constexpr int kTile = 64;                  // tokens per tile: a lane each
constexpr int kCus = 256;
constexpr int kAhead = 3;                  // operand steps in flight from LDS
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

// LDS place of a 16-byte chunk: chunk c of token t's row is stored at c ^ swz(t).
// Latent rows are multiples of 256 bytes, so their banks repeat every 16 chunks and
// swz runs over 16 values, tokens 0..7 on even ones (a transposing read takes chunk
// pairs of 8 tokens at a time); the 128-byte positional rows alternate between two
// halves of the banks, and 8 values over token pairs do.
template <int kChunks>
__device__ __forceinline__ int swz(int t) {
  if constexpr (kChunks >= 16) return (((t & 7) ^ (((t >> 3) & 1) << 2)) << 1) | ((t >> 3) & 1);
  return (t >> 1) & 7;
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
  int64_t ks;
  int window;
};

// False when the row belongs to no sequence.
__device__ __forceinline__ bool row_of(const AttnArgs& a, int64_t r, Row& o) {
  o.seq = a.row_seq ? a.row_seq[r] : (int)((uint32_t)r / (uint32_t)a.rows_per_seq);
  if (o.seq < 0 || o.seq >= a.B) return false;
  o.ks = a.ks ? a.ks[r] : 0;
  o.window = (int)min(max((int64_t)a.ke[r] - o.ks, (int64_t)0), a.max_tokens);
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
  const int64_t p = a.indices ? (int64_t)entry - row.ks : entry;
  return p >= 0 && p < row.window && (!a.indices || e < a.k) ? (int)p : -1;
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
  int pages;              // of the cache, at most 2^31 - 1: all that a table names
  uint32_t cache_bytes;   // the cache's size where it is below 4 GiB, and of a query row's heads
  uint32_t q_bytes;
};

// 16 bytes a lane to LDS, at dst + 16 * lane.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t rs, MXIDX_LDS uint8_t* dst, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (MXIDX_LDS void*)dst, 16, offset, 0, 0, 0);
}

// The copy of a tile's rows to LDS, kMine of them by each wave, in kPieces parts that
// the caller issues between its products: latent rows first, then the positional ones,
// C 16-byte chunks of each.  Lane t holds the cache byte of token t's row: where 32-bit
// offsets reach the whole cache (kSmall) as lo, and rows that fill less than an
// instruction share one; else as (lo, hi), with a descriptor and an instruction for each
// row.  A place without a row (kNoRow as lo, or as hi) is out of its descriptor's range
// and reads as zeros.
constexpr int64_t kReach = 0xfffe0000ll;   // of 32-bit offsets
constexpr int kNoRow = (int)0xffff0000u;   // past it, no wrap within a row; negative

template <int kLatent, int kMine, bool kSmall>
struct TileCopy {
  static constexpr int kRowBytes = (kLatent + kRopeWidth) * 2;
  static constexpr int LC = kLatent / 8, PC = kRopeWidth / 8;
  static constexpr int kLatentPer = LC >= kWave || !kSmall ? 1 : kWave / LC;
  static constexpr int kPosPer = kSmall ? kWave / PC : 1;
  static constexpr int kLatentPieces = kMine / kLatentPer, kPosPieces = kMine / kPosPer;
  static constexpr int kPieces = kLatentPieces + kPosPieces;
  static_assert(kMine % kLatentPer == 0 && kMine % kPosPer == 0, "whole instructions");

  template <int C, int kPer>
  static __device__ __forceinline__ void rows(const char* base, uint32_t bytes, MXIDX_LDS uint8_t* dst, int t0,
                                              int lo, int hi, int offset, int ln) {
    if constexpr (kSmall) {
      const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(base, (int)bytes);
      const int t = t0 + (kPer == 1 ? 0 : ln / C);
      const int row = kPer == 1 ? __builtin_amdgcn_readlane(lo, t) : __shfl(lo, t);
      copy16(rs, dst + t0 * C * 16, row + offset + (((ln % C) ^ swz<C>(t)) << 4));
    } else if (C >= kWave || ln < C) {
      const uint32_t l32 = (uint32_t)__builtin_amdgcn_readlane(lo, t0);
      const int h32 = __builtin_amdgcn_readlane(hi, t0);
      copy16(buffer_rsrc(base + (((uint64_t)(uint32_t)max(h32, 0) << 32) | l32), h32 < 0 ? 0 : kRowBytes),
             dst + __builtin_amdgcn_readfirstlane(t0 * C * 16),
             ((ln << 4) ^ __builtin_amdgcn_readfirstlane(swz<C>(t0) << 4)) + offset);
    }
  }

  // Piece i of the rows from `first` on.
  static __device__ __forceinline__ void piece(int i, const char* base, uint32_t bytes, MXIDX_LDS uint8_t* tile,
                                               int first, int lo, int hi, int ln) {
    if (i < kLatentPieces)
      rows<LC, kLatentPer>(base, bytes, tile, first + i * kLatentPer, lo, hi, 0, ln);
    else
      rows<PC, kPosPer>(base, bytes, tile + kTile * kLatent * 2, first + (i - kLatentPieces) * kPosPer, lo, hi,
                        kLatent * 2, ln);
  }
};

template <int kLatent, int HG, int TH, bool kSmall>
__global__ __launch_bounds__(HG * TH * kWave, 1) void attn_kernel(AttnArgs a, Parts parts) {
  constexpr int kRow = kLatent + kRopeWidth;
  constexpr int kWaves = HG * TH, kHeads = HG * 16;
  constexpr int kTokens = kTile / TH;                  // of a tile, per wave
  constexpr int NT = kTokens < 32 ? 1 : 2;             // 16-token parts of a step
  constexpr int KS = kRow / 32, KL = kLatent / 32;     // contraction steps, latent ones
  constexpr int NV = kLatent / 16;                     // 16-value parts of the output
  constexpr int LC = kLatent / 8;                      // 16-byte chunks of a latent row
  constexpr int kMine = kTile / kWaves;                // rows that a wave copies
  constexpr int kLatentBytes = kTile * kLatent * 2, kTileBytes = kTile * kRow * 2;
  using Copy = TileCopy<kLatent, kMine, kSmall>;
  constexpr int kSteps = kTokens / (16 * NT);          // of a wave's part of a tile
  // Two arrays, and the loop below unrolled over them: the compiler then sees that a
  // tile's reads do not touch the one being copied, and does not wait for its copies.
  __shared__ __attribute__((aligned(1024))) uint8_t tile0[kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t tile1[kTileBytes];
  static_assert(2 * kTileBytes <= 156 * 1024, "two tiles fit the LDS");
  __shared__ float2 stats[TH][kHeads];                 // the waves' (m, l), then the output's scale

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int hg = wave % HG, th = wave / HG;
  const uint32_t groups = (uint32_t)parts.heads / kHeads, unit = blockIdx.x / groups;
  const int group = (int)(blockIdx.x - unit * groups);
  const uint32_t r32 = unit / (uint32_t)parts.splits;
  const int split = (int)(unit - r32 * (uint32_t)parts.splits);
  const int64_t r = r32;
  Row row;
  if (!row_of(a, r, row)) return;
  const int entries = row.window == 0 ? 0 : a.indices ? a.k : row.window;
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

  // The lanes' cache rows of a tile as byte offsets, and which places hold a token.
  auto rows_of = [&](int p, int page, uint64_t& mask, int& lo, int& hi) __attribute__((always_inline)) {
    const bool ok = p >= 0 && page >= 0 && page < parts.pages;
    mask = __ballot(ok);
    const uint64_t mine = ((uint64_t)(uint32_t)page * kPage + (uint32_t)(p % kPage)) * (kRow * 2);
    lo = ok || !kSmall ? (int)(uint32_t)mine : kNoRow;
    hi = ok ? (int)(uint32_t)(mine >> 32) : kNoRow;
  };
  const char* cache = static_cast<const char*>(a.cache);

  // kTokens tokens of a tile against the wave's heads, 16 * NT at a time; the pieces of the
  // next tile's copy go between the steps of the first product
  auto compute = [&](MXIDX_LDS const uint8_t* buf, uint64_t mask, MXIDX_LDS uint8_t* nxt, int lo,
                     int hi) __attribute__((always_inline)) {
    // pieces of the copy in each step: the positional rows are in all of them (they are
    // few, and the same)
    constexpr int kL = Copy::kLatentPieces / kSteps, kP = kL + Copy::kPieces - Copy::kLatentPieces;
    int first = wave * kMine;                          // of the latent rows left to copy
    int stop = (th + 1) * kTokens;
    asm volatile("" : "+s"(stop));                     // stays a loop
#pragma unroll 1
    for (int base = th * kTokens; base < stop; base += 16 * NT) {
      v4f s[NT];
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
        v8s x[kAhead][NT];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) keys(k, x[k]);
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t = 0; t < NT; ++t) s[t] = mfma_bf16(x[k % kAhead][t], q[k], s[t]);
          if (k + kAhead < KS) keys(k + kAhead, x[k % kAhead]);
#pragma unroll
          for (int i = 0; i < kP; ++i)
            if (i * KS / kP == k)
              Copy::piece(i < kL ? i : Copy::kLatentPieces + i - kL, cache, parts.cache_bytes, nxt,
                          i < kL ? first : wave * kMine, lo, hi, ln);
        }
        first += kMine / kSteps;
        __builtin_amdgcn_sched_barrier(0);
      }
      // s[t][i]: token base + 16t + 4g + i of this lane's head
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] *= scale2;
      if (mask != ~0ull) {
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
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
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
      uint32_t w[NT][2];
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
      }
      // values: lane 4j + c of a 16-lane group reads tokens 4g + j, values 4c..4c+3, and
      // gets tokens 4g..4g+3 of value n
      const int vl = fresh_lane(), vn = vl & 15, vt = 4 * (vl >> 4) + (vn >> 2);
      const int val = (base + vt) * (kLatent * 2) + ((((vn >> 1) & 1) ^ swz<LC>(vt)) << 4) + 8 * (vn & 1);
      v4s y[kAhead][NT];
      auto values = [&](int v, v4s (&x)[NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          x[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MXIDX_LDS v4s*)(
              buf + (val ^ ((v & 7) << 5)) + (v >> 3) * 256 + t * 16 * (kLatent * 2)));
      };
#pragma unroll
      for (int v = 0; v < kAhead; ++v) values(v, y[v]);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        __builtin_amdgcn_sched_barrier(0);
        const v4s(&z)[NT] = y[v % kAhead];
        if constexpr (NT == 1)
          o[v] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(z[0], __builtin_bit_cast(v4s, uint2{w[0][0], w[0][1]}),
                                                            o[v], 0, 0, 0);
        else
          o[v] = mfma_bf16(__builtin_shufflevector(z[0], z[NT - 1], 0, 1, 2, 3, 4, 5, 6, 7),
                           __builtin_bit_cast(v8s, uint4{w[0][0], w[0][1], w[NT - 1][0], w[NT - 1][1]}), o[v]);
        if (v + kAhead < NV) values(v + kAhead, y[v % kAhead]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // the pipeline: the tile computed, the next one's rows on their way to LDS, the one
  // behind it looking up its pages and the one behind that its list entries
  if (t0 < t1) {
    auto place = [&](int t) { return t * kTile + fresh_lane(); };
    auto entry = [&](int t) { return list_entry(a, r, place(min(t, t1 - 1))); };
    const int e0 = entry(t0), e1 = entry(t0 + 1);
    int far = entry(t0 + 2);
    const int now = token_of(a, row, e0, place(t0));
    const int now_page = token_page(a, row, now);
    int next = token_of(a, row, e1, place(t0 + 1));
    int page = token_page(a, row, next);
    uint64_t mask;
    int lo, hi;
    auto copy_all = [&](const char* base, uint32_t bytes, MXIDX_LDS uint8_t* tile) __attribute__((always_inline)) {
      const int ln = fresh_lane();
#pragma unroll
      for (int i = 0; i < Copy::kPieces; ++i) Copy::piece(i, base, bytes, tile, wave * kMine, lo, hi, ln);
    };
    // the query's rows, as if they were a tile's, to LDS: 64 heads to tile1 behind the
    // list's and pages' loads, and with 128 heads the others to tile0 before the tile
    constexpr int kQTiles = (kHeads + kTile - 1) / kTile;
#pragma unroll
    for (int i = 0; i < kQTiles; ++i) {
      const int h = i * kTile + fresh_lane(), head = group * kHeads + h;
      const uint64_t at = (uint64_t)min(head, a.H - 1) * (uint64_t)a.q_head_stride * 2;
      const bool ok = h < kHeads && head < a.H;
      lo = ok || !kSmall ? (int)(uint32_t)at : kNoRow;
      hi = ok ? (int)(uint32_t)(at >> 32) : kNoRow;
      copy_all(static_cast<const char*>(a.q) + r * a.q_row_stride * 2, parts.q_bytes,
               (MXIDX_LDS uint8_t*)(i == 0 ? tile1 : tile0));
    }
    rows_of(now, now_page, mask, lo, hi);
    if (kQTiles == 1) copy_all(cache, parts.cache_bytes, (MXIDX_LDS uint8_t*)tile0);
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
      copy_all(cache, parts.cache_bytes, (MXIDX_LDS uint8_t*)tile0);
    }
    // tile t from `cur`, tile t + 1 on its way to `nxt` (behind the last one: zeros)
    auto step = [&](int t, MXIDX_LDS uint8_t* cur, MXIDX_LDS uint8_t* nxt) __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      uint64_t next_mask;
      rows_of(t + 1 < t1 ? next : -1, page, next_mask, lo, hi);
      next = token_of(a, row, far, place(t + 2));
      page = token_page(a, row, next);
      far = entry(t + 3);
      seen |= mask != 0;
      compute(cur, mask, nxt, lo, hi);
      mask = next_mask;
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
  constexpr int kValues = HG == 8 ? kLatent / 2 : kLatent;
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

// The splits' sums of one (row, head), kLatent / 4 lanes: 4 values each, the loads of
// kBatch splits together.
constexpr int kBatch = 8;
template <int kLatent>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Parts parts) {
  constexpr int W = kLatent / 4;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / W;
  const int i = threadIdx.x % W;
  const int64_t r = (uint32_t)at / (uint32_t)a.H;      // rows * H < 2^31
  const int head = (int)(at - r * a.H);
  Row row;
  if (r >= a.rows || !row_of(a, r, row)) return;
  const int64_t first = r * parts.splits * parts.heads + head;
  v4f o = {0.f, 0.f, 0.f, 0.f};
  float top = neg_inf(), l = 0.f;
  for (int s0 = 0; s0 < parts.splits; s0 += kBatch) {
    float2 ml[kBatch];
    v4f x[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int64_t p = first + (int64_t)min(s0 + s, parts.splits - 1) * parts.heads;
      ml[s] = *reinterpret_cast<const float2*>(parts.ml + 2 * p);
      x[s] = *reinterpret_cast<const v4f*>(parts.o + p * kLatent + 4 * i);
    }
    float m = top;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) m = fmaxf(m, ml[s].x);
    const float ref = m == neg_inf() ? 0.f : m;
    const float old = __builtin_amdgcn_exp2f(top - ref);
    o *= old;
    l *= old;
    top = m;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      if (s0 + s >= parts.splits || ml[s].y == 0.f) continue;   // nothing seen: no sums written
      const float f = __builtin_amdgcn_exp2f(ml[s].x - ref);
      l += f * ml[s].y;
      o += f * x[s];
    }
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
  int heads;              // H rounded up to whole groups
  int splits;
};

Plan plan_of(int64_t rows, int H, int64_t entries) {
  Plan p;
  p.group_heads = H <= 16 ? 16 : H <= 32 ? 32 : H <= 64 ? 64 : 128;
  p.heads = (H + p.group_heads - 1) / p.group_heads * p.group_heads;
  const int64_t units = rows * (p.heads / p.group_heads);
  const int64_t tiles = (entries + kTile - 1) / kTile;
  int64_t s = units > 0 ? kCus / units : 1;
  s = s < tiles ? s : tiles;
  p.splits = (int)(s > 1 ? s : 1);
  return p;
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

int64_t ml_bytes(int64_t rows, const Plan& p) { return align256(rows * p.splits * p.heads * 8); }

template <int kLatent>
hipError_t launch(const AttnArgs& a, void* workspace, hipStream_t stream) {
  const Plan p = plan_of(a.rows, a.H, a.indices ? a.k : a.max_tokens);
  const int64_t cache_bytes = a.num_pages * kPage * (kLatent + kRopeWidth) * 2;
  const int64_t q_bytes = ((a.H - 1) * a.q_head_stride + kLatent + kRopeWidth) * 2;
  const bool small = cache_bytes <= kReach && q_bytes <= kReach;
  Parts parts{nullptr, nullptr, p.splits, p.heads, (int)(a.num_pages < 0x7fffffff ? a.num_pages : 0x7fffffff),
              small ? (uint32_t)cache_bytes : 0, small ? (uint32_t)q_bytes : 0};
  if (p.splits > 1) {
    parts.ml = static_cast<float*>(workspace);
    parts.o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(a.rows, p));
  }
  const dim3 grid((uint32_t)(a.rows * (p.heads / p.group_heads) * p.splits));
#define MXIDX_ATTN(heads_, hg, th)                                                              \
  case heads_:                                                                                  \
    if (small)                                                                                  \
      hipLaunchKernelGGL((attn_kernel<kLatent, hg, th, true>), grid, dim3(hg * th * kWave), 0,  \
                         stream, a, parts);                                                     \
    else                                                                                        \
      hipLaunchKernelGGL((attn_kernel<kLatent, hg, th, false>), grid, dim3(hg * th * kWave), 0, \
                         stream, a, parts);                                                     \
    break;
  switch (p.group_heads) {
    MXIDX_ATTN(16, 1, 4)
    MXIDX_ATTN(32, 2, 2)
    MXIDX_ATTN(64, 4, 2)
    MXIDX_ATTN(128, 8, 1)
    default: return hipErrorInvalidValue;
  }
#undef MXIDX_ATTN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  constexpr int W = kLatent / 4;
  const int64_t threads = a.rows * a.H * W;
  hipLaunchKernelGGL(attn_join_kernel<kLatent>, dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0,
                     stream, a, parts);
  return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t rows, int H, int latent, int64_t entries) {
  const Plan p = plan_of(rows, H, entries);
  if (p.splits == 1) return 0;
  return ml_bytes(rows, p) + rows * p.splits * p.heads * latent * 4;
}

hipError_t launch_attn_paged(const AttnArgs& a, int latent, void* workspace, hipStream_t stream) {
  switch (latent) {
    case 128: return launch<128>(a, workspace, stream);
    case 256: return launch<256>(a, workspace, stream);
    default: return launch<512>(a, workspace, stream);
  }
}

}  // namespace mxidx
