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
  if constexpr (kChunks >= 16) return ((t & 7) << 1) | ((t >> 3) & 1);
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
  uint32_t cache_bytes;   // the cache's size below 4 GiB (small_cache)
  bool small_cache;
};

// 16 bytes a lane to LDS, at dst + 16 * lane.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t rs, MXIDX_LDS uint8_t* dst, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (MXIDX_LDS void*)dst, 16, offset, 0, 0, 0);
}

// Copies C 16-byte chunks, from byte `offset` on, of each of kMine rows of a tile to
// LDS: token t = first .. first + kMine - 1 from the cache row whose byte lane t holds
// (lo, hi).  Rows that fill less than an instruction share one where 32-bit offsets
// reach the whole cache, and take one each where they do not.
template <int C, int kMine, int kRowBytes>
__device__ __forceinline__ void copy_rows(const char* base, const Parts& parts, MXIDX_LDS uint8_t* dst,
                                          int first, int lo, int hi, int offset, int ln) {
  constexpr int kPer = C >= kWave ? 1 : kWave / C;
  static_assert(C <= kWave && kMine % kPer == 0, "whole instructions");
  if (kPer > 1 && parts.small_cache) {
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(base, (int)parts.cache_bytes);
#pragma unroll
    for (int i = 0; i < kMine; i += kPer) {
      const int t = first + i + ln / C;
      copy16(rs, dst + (first + i) * C * 16, __shfl(lo, t) + offset + (((ln % C) ^ swz<C>(t)) << 4));
    }
  } else if (kPer == 1 || ln < C) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int t = first + i;
      const uint32_t l32 = (uint32_t)__builtin_amdgcn_readlane(lo, t);
      const uint32_t h32 = (uint32_t)__builtin_amdgcn_readlane(hi, t);
      copy16(buffer_rsrc(base + (((uint64_t)h32 << 32) | l32), kRowBytes), dst + t * C * 16,
             offset + ((ln ^ swz<C>(t)) << 4));
      __builtin_amdgcn_sched_barrier(0);               // one row's descriptor at a time
    }
  }
}

template <int kLatent, int HG, int MT, int TH>
__global__ __launch_bounds__(HG * TH * kWave, 1) void attn_kernel(AttnArgs a, Parts parts) {
  constexpr int kRow = kLatent + kRopeWidth;
  constexpr int kWaves = HG * TH;
  constexpr int kHeads = HG * MT * 16;                 // of the workgroup
  constexpr int kTokens = kTile / TH;                  // of a tile, per wave
  constexpr int NT = kTokens < 32 ? 1 : 2;             // 16-token parts of a step
  constexpr int KS = kRow / 32, KL = kLatent / 32;     // contraction steps, latent ones
  constexpr int NV = kLatent / 16;                     // 16-value parts of the output
  constexpr int LC = kLatent / 8;                      // 16-byte chunks of a latent row
  constexpr int kLatentBytes = kTile * kLatent * 2, kTileBytes = kTile * kRow * 2;
  // Two arrays, and the loop below unrolled over them: the compiler then sees that a
  // tile's reads do not touch the one being copied, and does not wait for its copies.
  __shared__ __attribute__((aligned(1024))) uint8_t tile0[kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t tile1[kTileBytes];
  static_assert(2 * kTileBytes <= 160 * 1024, "two tiles fit the LDS");
  constexpr int kJoin = 16 * kLatent * 4;              // a wave's 16 heads, joined at the end
  constexpr int kJoin0 = kTileBytes / kJoin;           // of them in the first tile
  static_assert((TH - 1) * HG <= 2 * kJoin0, "the waves' join fits the tiles");
  __shared__ float join_ml[TH > 1 ? TH * kHeads * 2 : 1];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int hg = wave % HG, th = wave / HG;
  const int g = lane >> 4, n = lane & 15;
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
  const int head0 = group * kHeads + hg * MT * 16 + n; // this lane's heads: head0 + 16u

  // the wave's query: step s holds values 32s + 8g .. +7 of a head
  v8s q[MT][KS];
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + r * a.q_row_stride +
                        (int64_t)min(head0 + 16 * u, a.H - 1) * a.q_head_stride + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) q[u][s] = *reinterpret_cast<const v8s*>(p + 32 * s);
  }
  v4f o[MT][NV];
  float m[MT], l[MT];                                  // l: this lane's tokens only
#pragma unroll
  for (int u = 0; u < MT; ++u) {
#pragma unroll
    for (int v = 0; v < NV; ++v) o[u][v] = v4f{0.f, 0.f, 0.f, 0.f};
    m[u] = neg_inf();
    l[u] = 0.f;
  }
  const float scale2 = a.scale * 1.4426950408889634f;  // scores in powers of two

  // Copies the tile's rows, kTile/kWaves by each wave: lane i holds the cache row of
  // token i.  By buffer loads: the compiler counts them apart from the LDS reads, which
  // it would drain at every use behind global_load_lds's.  Nothing of it is kept over the
  // products: they take all registers, and a spilled one would be waited for behind the
  // copies.
  auto stage = [&](MXIDX_LDS uint8_t* buf, int64_t cache_row) __attribute__((always_inline)) {
    constexpr int kMine = kTile / kWaves;
    const int first = wave * kMine;
    const char* base = static_cast<const char*>(a.cache);
    const uint64_t bytes = (uint64_t)cache_row * (kRow * 2);
    const int lo = (int)(uint32_t)bytes, hi = (int)(uint32_t)(bytes >> 32);
    const int ln = fresh_lane();
    copy_rows<LC, kMine, kRow * 2>(base, parts, buf, first, lo, hi, 0, ln);
    copy_rows<8, kMine, kRow * 2>(base, parts, buf + kLatentBytes, first, lo, hi, kLatent * 2, ln);
  };
  // The lanes' cache rows of a tile; places of no token take the first visible one's.
  auto rows_of = [&](int p, int page, uint64_t& mask) -> int64_t {
    const bool ok = p >= 0 && page >= 0 && page < parts.pages;
    mask = __ballot(ok);
    const int64_t mine = (int64_t)page * kPage + p % kPage;
    const int from = ok || mask == 0 ? fresh_lane() : __builtin_ctzll(mask);
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)mine, from);
    const uint32_t hi = (uint32_t)__shfl((int)(uint32_t)((uint64_t)mine >> 32), from);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  };

  // kTokens tokens of a tile against the wave's heads, 16 * NT at a time
  auto compute = [&](MXIDX_LDS const uint8_t* buf, uint64_t mask) __attribute__((always_inline)) {
    int stop = (th + 1) * kTokens;
    asm volatile("" : "+s"(stop));                     // stays a loop
#pragma unroll 1
    for (int base = th * kTokens; base < stop; base += 16 * NT) {
      // LDS offsets of the operands in the tile: the places of the chunks differ between
      // steps by constants xored into few bits (swz), so one register for each kind of
      // row does
      const int ln = fresh_lane(), n = ln & 15, g = ln >> 4;
      const int key = base * (kLatent * 2) + n * (kLatent * 2) + ((g ^ swz<LC>(n)) << 4);
      const int pos = kLatentBytes + base * (kRopeWidth * 2) + n * (kRopeWidth * 2) + ((g ^ swz<8>(n)) << 4);
      v4f s[MT][NT];
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[u][t] = v4f{0.f, 0.f, 0.f, 0.f};
      // keys: kAhead steps are on their way while one is used
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
      for (int k = 0; k < KS; ++k) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < MT; ++u) s[u][t] = mfma_bf16(x[k % kAhead][t], q[u][k], s[u][t]);
        if (k + kAhead < KS) keys(k + kAhead, x[k % kAhead]);
      }
      __builtin_amdgcn_sched_barrier(0);
      // s[u][t][i]: token base + 16t + 4g + i, head head0 + 16u
      float f[MT];
      bool grow = false;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        float top = neg_inf();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][t][i] *= scale2;
        if (mask != ~0ull) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t bits = (uint32_t)(mask >> (base + 16 * t + 4 * (fresh_lane() >> 4)));
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][t][i] = (bits >> i) & 1 ? s[u][t][i] : neg_inf();
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[u][t][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // the reference is raised only where weights would pass 2^kSlack: what was summed
        // so far is seldom rescaled
        f[u] = 1.f;
        if (m[u] == neg_inf()) {
          m[u] = top;                                  // nothing summed yet
        } else if (top > m[u] + kSlack) {
          f[u] = __builtin_amdgcn_exp2f(m[u] - top);
          m[u] = top;
          grow = true;
        }
      }
      if (__any(grow)) {
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          l[u] *= f[u];
#pragma unroll
          for (int v = 0; v < NV; ++v) o[u][v] *= f[u];
        }
      }
      uint32_t w[MT][NT][2];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const float ref = m[u] == neg_inf() ? 0.f : m[u];   // no token yet: every weight 0
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = __builtin_amdgcn_exp2f(s[u][t][i] - ref);
            l[u] += p[i];
          }
          w[u][t][0] = pack2(p[0], p[1]);
          w[u][t][1] = pack2(p[2], p[3]);
        }
      }
      // values: lane 4j + c of a 16-lane group reads tokens 4g + j, values 4c..4c+3, and
      // gets tokens 4g..4g+3 of value n
      const int vl = fresh_lane(), vn = vl & 15, vt = 4 * (vl >> 4) + (vn >> 2);
      const int val = base * (kLatent * 2) + vt * (kLatent * 2) +
                      ((((vn >> 1) & 1) ^ swz<LC>(vt)) << 4) + 8 * (vn & 1);
      v4s y[kAhead][NT];
      auto values = [&](int v, v4s (&r)[NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          r[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MXIDX_LDS v4s*)(
              buf + (val ^ ((v & 7) << 5)) + (v >> 3) * 256 + t * 16 * (kLatent * 2)));
      };
#pragma unroll
      for (int v = 0; v < kAhead; ++v) values(v, y[v]);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        __builtin_amdgcn_sched_barrier(0);
        const v4s(&z)[NT] = y[v % kAhead];
        if constexpr (NT == 1) {
#pragma unroll
          for (int u = 0; u < MT; ++u)
            o[u][v] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                z[0], __builtin_bit_cast(v4s, uint2{w[u][0][0], w[u][0][1]}), o[u][v], 0, 0, 0);
        } else {
          const v8s zz = __builtin_shufflevector(z[0], z[NT - 1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int u = 0; u < MT; ++u)
            o[u][v] = mfma_bf16(zz, __builtin_bit_cast(v8s, uint4{w[u][0][0], w[u][0][1], w[u][NT - 1][0],
                                                                  w[u][NT - 1][1]}), o[u][v]);
        }
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
    uint64_t mask;
    {
      const int now = token_of(a, row, entry(t0), place(t0));
      const int64_t rows = rows_of(now, token_page(a, row, now), mask);
      if (mask) stage((MXIDX_LDS uint8_t*)tile0, rows);
    }
    int next = token_of(a, row, entry(t0 + 1), place(t0 + 1));
    int page = token_page(a, row, next);
    int far = entry(t0 + 2);
    // tile t from `cur`, tile t + 1 on its way to `nxt`
    auto step = [&](int t, MXIDX_LDS uint8_t* cur, MXIDX_LDS uint8_t* nxt) __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      uint64_t next_mask = 0;
      if (t + 1 < t1) {
        const int64_t rows = rows_of(next, page, next_mask);
        if (next_mask) stage(nxt, rows);
        next = token_of(a, row, far, place(t + 2));
        page = token_page(a, row, next);
        far = entry(t + 3);
      }
      if (mask) compute(cur, mask);
      mask = next_mask;
    };
    for (int t = t0; t < t1; t += 2) {
      step(t, (MXIDX_LDS uint8_t*)tile0, (MXIDX_LDS uint8_t*)tile1);
      if (t + 1 < t1) step(t + 1, (MXIDX_LDS uint8_t*)tile1, (MXIDX_LDS uint8_t*)tile0);
    }
  }

#pragma unroll
  for (int u = 0; u < MT; ++u) {
    l[u] += __shfl_xor(l[u], 16);
    l[u] += __shfl_xor(l[u], 32);
  }
  if constexpr (TH > 1) {
    // the token parts' sums joined in LDS, 16 heads at a time: part th > 0 leaves its
    // own, part 0 takes them
    auto place = [&](int i) {                          // of the i-th leaving wave
      return reinterpret_cast<float*>(i < kJoin0 ? tile0 + i * kJoin : tile1 + (i - kJoin0) * kJoin) + 4 * lane;
    };
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      const int slot = (th * HG + hg) * MT * 16 + 16 * u + n;
      if (g == 0) {
        join_ml[2 * slot] = m[u];
        join_ml[2 * slot + 1] = l[u];
      }
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      __syncthreads();                                 // the last reads are done
      if (th > 0) {
        float* dst = place((th - 1) * HG + hg);
#pragma unroll
        for (int v = 0; v < NV; ++v) *reinterpret_cast<v4f*>(dst + v * 256) = o[u][v];
      }
      __syncthreads();
      if (th > 0) continue;
      float top = m[u];
#pragma unroll
      for (int t = 1; t < TH; ++t)
        top = fmaxf(top, join_ml[2 * ((t * HG + hg) * MT * 16 + 16 * u + n)]);
      const float ref = top == neg_inf() ? 0.f : top;
      float f = __builtin_amdgcn_exp2f(m[u] - ref);
      l[u] *= f;
#pragma unroll
      for (int v = 0; v < NV; ++v) o[u][v] *= f;
#pragma unroll
      for (int t = 1; t < TH; ++t) {
        const int slot = (t * HG + hg) * MT * 16 + 16 * u + n;
        f = __builtin_amdgcn_exp2f(join_ml[2 * slot] - ref);
        l[u] += f * join_ml[2 * slot + 1];
        const float* src = place((t - 1) * HG + hg);
#pragma unroll
        for (int v = 0; v < NV; ++v) o[u][v] += f * *reinterpret_cast<const v4f*>(src + v * 256);
      }
      m[u] = top;
    }
    if (th > 0) return;
  }

  // o[u][v][i]: value 16v + 4g + i of head head0 + 16u
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int head = head0 + 16 * u;
    if (parts.splits > 1) {
      const int64_t at = (r * parts.splits + split) * parts.heads + head;
      if (g == 0) *reinterpret_cast<float2*>(parts.ml + 2 * at) = make_float2(m[u], l[u]);
      if (__all(l[u] == 0.f)) continue;
      float* dst = parts.o + at * kLatent + 4 * g;
#pragma unroll
      for (int v = 0; v < NV; ++v) *reinterpret_cast<v4f*>(dst + 16 * v) = o[u][v];
      continue;
    }
    if (head >= a.H) continue;
    const float inv = l[u] == 0.f ? 0.f : 1.f / l[u];
    uint16_t* out = static_cast<uint16_t*>(a.out) + r * a.out_row_stride +
                    (int64_t)head * a.out_head_stride + 4 * g;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      *reinterpret_cast<uint2*>(out + 16 * v) =
          make_uint2(pack2(o[u][v][0] * inv, o[u][v][1] * inv), pack2(o[u][v][2] * inv, o[u][v][3] * inv));
    if (a.lse && g == 0)
      a.lse[r * a.H + head] = l[u] == 0.f ? neg_inf() : m[u] * 0.6931471805599453f + logf(l[u]);
  }
}

// The splits' sums of one (row, head), kLatent / 4 lanes: 4 values each.
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
  float top = neg_inf();
  for (int s = 0; s < parts.splits; ++s)
    top = fmaxf(top, parts.ml[2 * (first + (int64_t)s * parts.heads)]);
  v4f o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  for (int s = 0; s < parts.splits; ++s) {
    const int64_t p = first + (int64_t)s * parts.heads;
    const float2 ml = *reinterpret_cast<const float2*>(parts.ml + 2 * p);
    if (ml.y == 0.f) continue;                         // nothing seen: no sums written
    const float f = __builtin_amdgcn_exp2f(ml.x - top);
    l += f * ml.y;
    o += f * *reinterpret_cast<const v4f*>(parts.o + p * kLatent + 4 * i);
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
  const bool small = cache_bytes < (1ll << 32);
  Parts parts{nullptr, nullptr, p.splits, p.heads, (int)(a.num_pages < 0x7fffffff ? a.num_pages : 0x7fffffff),
              small ? (uint32_t)cache_bytes : 0, small};
  if (p.splits > 1) {
    parts.ml = static_cast<float*>(workspace);
    parts.o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(a.rows, p));
  }
  const dim3 grid((uint32_t)(a.rows * (p.heads / p.group_heads) * p.splits));
  switch (p.group_heads) {
    case 16: hipLaunchKernelGGL((attn_kernel<kLatent, 1, 1, 4>), grid, dim3(256), 0, stream, a, parts); break;
    case 32: hipLaunchKernelGGL((attn_kernel<kLatent, 2, 1, 2>), grid, dim3(256), 0, stream, a, parts); break;
    case 64: hipLaunchKernelGGL((attn_kernel<kLatent, 4, 1, 2>), grid, dim3(512), 0, stream, a, parts); break;
    default: hipLaunchKernelGGL((attn_kernel<kLatent, 8, 1, 1>), grid, dim3(512), 0, stream, a, parts); break;
  }
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
