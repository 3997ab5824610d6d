// A serving step's bookkeeping from its request lengths (idx_step_map): which
// request each of the step's rows belongs to, its position, slot and window, and
// the block-table entries of the pages that the step enters.
//
// With L_b tokens of which Q_b are new, request b held h_b = ceil((L_b - Q_b)/64)
// pages, its rows begin at row sum_{b'<b} Q_b', the pages it enters are
// ceil(L_b/64) - h_b entries of the free list from sum_{b'<b} of the same on, and
// its gathered K begins at row sum_{b'<b} L_b'.
//
// Work mapping: one thread per row of the step, 256 rows of a workgroup at a time.  Every
// workgroup takes the three prefix sums over all requests itself (each thread a run of
// consecutive requests, then one scan over the workgroup), so one launch does, with no
// workspace and no order between workgroups.  The thread that owns a request with rows among the
// workgroup's rows marks its first one there; a running maximum over the rows then
// gives each row its request.  A page that the step enters is entered by exactly one
// of its rows (the one at a multiple of 64), whose thread writes the table
// entry; table entries are read only below h_b and written only from h_b on.
//
// Bound by latency: 16 requests move under a kilobyte (3.4 us; 4096 of one row 12.0), and
// the largest steps 28 bytes a row (64 requests, 1 M rows: 12.5 us; 4096 requests, 2 M
// rows: 70 us, most of it the requests' sums in each workgroup).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace mxidx {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct Sums {
  int64_t q, pages, tokens;   // new tokens, pages entered, tokens
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.q + b.q, a.pages + b.pages, a.tokens + b.tokens};
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const uint32_t lo = __shfl_up((uint32_t)v, d);
  const uint32_t hi = __shfl_up((uint32_t)((uint64_t)v >> 32), d);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens) {
  return tokens <= 0 ? 0 : (tokens + kPage - 1) / kPage;
}

struct Request {
  int64_t len, q;
  __device__ __forceinline__ int64_t before() const { return len - q; }
  __device__ __forceinline__ int64_t held() const { return pages_of(len - q); }
  __device__ __forceinline__ Sums sums() const { return {q, pages_of(len) - held(), len}; }
};

__device__ __forceinline__ Request request(const StepMapArgs& a, int b) {
  return {(int64_t)max(a.seq_lens[b], 0), (int64_t)max(a.query_lens[b], 0)};
}

// kAhead: requests of a thread's run that are loaded together; the run's first ones stay in
// registers.
template <int kAhead>
__global__ __launch_bounds__(kThreads) void step_map_kernel(StepMapArgs a) {
  __shared__ Sums wave_sum[kWaves];
  __shared__ int wave_mark[kWaves];
  __shared__ int mark[kThreads];             // request of the row, at the request's first row here
  __shared__ int64_t first_row[kThreads], entered[kThreads], gathered[kThreads];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;

  // this thread's requests, and the sums before them
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  Request first[kAhead];
  if (b0 < b1) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) first[i] = request(a, min(b0 + i, b1 - 1));
  }
  // f(b, request) for each of the run
  auto run = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (b0 + i < b1) f(b0 + i, first[i]);
    for (int b = b0 + kAhead; b < b1; b += kAhead) {
      Request r[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) r[i] = request(a, min(b + i, b1 - 1));
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (b + i < b1) f(b + i, r[i]);
    }
  };
  Sums own = {0, 0, 0};
  run([&](int, const Request& r) { own = own + r.sums(); });
  Sums incl = own;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const Sums up = {shfl_up64(incl.q, d), shfl_up64(incl.pages, d), shfl_up64(incl.tokens, d)};
    if (lane >= d) incl = incl + up;
  }
  if (lane == kWave - 1) wave_sum[wave] = incl;
  __syncthreads();
  Sums at = {incl.q - own.q, incl.pages - own.pages, incl.tokens - own.tokens};
  Sums total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at = at + wave_sum[w];
    total = total + wave_sum[w];
  }
  const int64_t free0 = a.free_pages ? a.free_start[0] : 0;
  if (blockIdx.x == 0 && tid == 0) {
    if (a.free_next) a.free_next[0] = free0 + total.pages;
    if (a.cu_seq_offsets) a.cu_seq_offsets[a.B] = total.tokens;
  }
  // the requests' offsets, spread over the workgroups
  if (a.cu_seq_offsets && tid % gridDim.x == blockIdx.x) {
    int64_t tokens = at.tokens;
    run([&](int b, const Request& r) {
      a.cu_seq_offsets[b] = tokens;
      tokens += r.len;
    });
  }

  for (int64_t row0 = (int64_t)blockIdx.x * kThreads; row0 < a.num_rows;
       row0 += (int64_t)gridDim.x * kThreads) {
    __syncthreads();                           // the rows before have read theirs
    mark[tid] = -1;
    __syncthreads();
    if (at.q < row0 + kThreads && at.q + own.q > row0) {
      Sums to = at;
      run([&](int b, const Request& r) {
        if (r.q > 0 && to.q < row0 + kThreads && to.q + r.q > row0) {
          const int i = (int)max(to.q - row0, (int64_t)0);
          mark[i] = b;
          first_row[i] = to.q;
          entered[i] = to.pages;
          gathered[i] = to.tokens;
        }
        to = to + r.sums();
      });
    }
    __syncthreads();

    // the last mark at or before this row
    int src = mark[tid] >= 0 ? tid : -1;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int up = __shfl_up(src, d);
      if (lane >= d) src = max(src, up);
    }
    if (lane == kWave - 1) wave_mark[wave] = src;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < wave) src = max(src, wave_mark[w]);

    const int64_t row = row0 + tid;
    if (row >= a.num_rows) continue;           // the last rows: no barrier follows
    int64_t pos = 0, slot = -1, col = 0;
    int seq = -1;
    if (row < total.q) {
      seq = mark[src];
      const Request r = request(a, seq);
      pos = r.before() + (row - first_row[src]);
      col = a.gathered ? gathered[src] : 0;
      const int64_t page = pos / kPage;
      if (pos >= 0 && page < a.bt_pages) {
        const int64_t held = r.held();
        int32_t id;
        if (a.free_pages && page >= held) {
          const int64_t f = free0 + entered[src] + (page - held);
          id = f >= 0 && f < a.num_free ? a.free_pages[f] : -1;
          if (a.block_table && pos % kPage == 0) a.block_table[seq * a.bt_row_stride + page] = id;
        } else {
          id = a.block_table ? a.block_table[seq * a.bt_row_stride + page] : -1;
        }
        if (id >= 0) slot = (int64_t)id * kPage + pos % kPage;
      }
    }
    if (a.slot_mapping) a.slot_mapping[row] = slot;
    if (a.positions) a.positions[row] = pos;
    if (a.row_seq) a.row_seq[row] = seq;
    if (a.ks) a.ks[row] = (int32_t)col;
    if (a.ke) a.ke[row] = seq < 0 ? 0 : (int32_t)(col + pos + 1);
  }
}

}  // namespace

// Four workgroups a CU take all rows between them, so that the requests' sums are taken that
// often at most (4096 requests, 2 M rows: 62 us, 73 with 2048, 134 with 8192 as with 256; 64
// requests, 1 M rows: 13.1, 14.1, 16.1 and 26.4).
constexpr int64_t kMaxBlocks = 1024;

hipError_t launch_step_map(const StepMapArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.num_rows + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)std::clamp<int64_t>(blocks, 1, kMaxBlocks));
  // as many requests together as a thread has, up to 8 (1024 requests: 5.0 us with 4, 6.0
  // with 8; 16 requests: 3.4 with 1, 3.75 with 8; 65535: 130 with 8, 240 one by one)
  if (a.B <= kThreads)
    hipLaunchKernelGGL(step_map_kernel<1>, grid, dim3(kThreads), 0, stream, a);
  else if (a.B <= 4 * kThreads)
    hipLaunchKernelGGL(step_map_kernel<4>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(step_map_kernel<8>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace mxidx
