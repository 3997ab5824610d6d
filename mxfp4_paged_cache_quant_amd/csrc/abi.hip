// C ABI of the MXFP4 indexer-cache library (declared in include/mxidx.h):
// host-side argument validation, the fail-closed gfx950 gate, and dispatch to
// the kernel launchers.  No allocation, no synchronization, no exceptions.
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "mxidx.h"
#include "launch.hpp"

static_assert(IDX_TOPK_NOALLOC_MAX_WORKSPACE == mxidx::kNoAllocScratchBytes,
              "the header's scratch limit is the size of the library's scratch array");

extern "C" int idx_arch_supported(const char* gcn_arch_name);

namespace {

constexpr int kMaxDevices = 64;
// 0 = not checked yet, 1 = gfx950, 2 = another architecture
std::atomic<int> g_gate[kMaxDevices];

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int gate_device(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return IDX_ERR_NO_DEVICE;
  const int st = g_gate[dev].load(std::memory_order_acquire);
  if (st == 1) return IDX_OK;
  if (st == 2) return IDX_ERR_UNSUPPORTED_ARCH;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return IDX_ERR_NO_DEVICE;
  const char* arch = prop.gcnArchName;
  // Test hook: pretend the device reports another architecture.
  if (const char* forced = std::getenv("MXIDX_FORCE_ARCH")) arch = forced;
  const bool ok = idx_arch_supported(arch) == IDX_OK;
  g_gate[dev].store(ok ? 1 : 2, std::memory_order_release);
  return ok ? IDX_OK : IDX_ERR_UNSUPPORTED_ARCH;
}

int gate_current() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return IDX_ERR_NO_DEVICE;
  if (dev >= 0 && dev < kMaxDevices && g_gate[dev].load(std::memory_order_acquire) == 1)
    return IDX_OK;                             // the common call: nothing more is asked
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) return IDX_ERR_NO_DEVICE;
  return gate_device(dev);
}

int launched(hipError_t e) { return e == hipSuccess ? IDX_OK : IDX_ERR_LAUNCH; }

bool heads_ok(int H) { return H >= 16 && H <= IDX_MAX_HEADS && H % 16 == 0; }

int check_rows_input(const void* x, int dtype, int64_t rows, int64_t row_stride) {
  if (rows < 0) return IDX_ERR_ARG;
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!x || !aligned(x, 16)) return IDX_ERR_ARG;
  if (row_stride < IDX_HEAD_DIM) return IDX_ERR_ARG;
  if (row_stride % (dtype == IDX_BF16 ? 8 : 4) != 0) return IDX_ERR_ARG;
  return IDX_OK;
}

}  // namespace

extern "C" {

int idx_version(void) { return 107; }

int idx_arch_supported(const char* gcn_arch_name) {
  // "gfx950" alone or followed by target features ("gfx950:sramecc+:xnack-")
  if (!gcn_arch_name) return IDX_ERR_UNSUPPORTED_ARCH;
  const bool ok = std::strncmp(gcn_arch_name, "gfx950", 6) == 0 &&
                  (gcn_arch_name[6] == '\0' || gcn_arch_name[6] == ':');
  return ok ? IDX_OK : IDX_ERR_UNSUPPORTED_ARCH;
}

const char* idx_strerror(int status) {
  switch (status) {
    case IDX_OK: return "ok";
    case IDX_ERR_ARG: return "invalid argument";
    case IDX_ERR_NO_DEVICE: return "no HIP device";
    case IDX_ERR_UNSUPPORTED_ARCH: return "device is not gfx950 (MI355X)";
    case IDX_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
  }
}

int idx_init(int device) {
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || device < 0 || device >= count)
    return IDX_ERR_NO_DEVICE;
  return gate_device(device);
}

int idx_quantize(const void* x, int dtype, int64_t rows, int64_t row_stride, uint8_t* values,
                 uint8_t* scales, hipStream_t stream) {
  int st = check_rows_input(x, dtype, rows, row_stride);
  if (st != IDX_OK) return st;
  if (rows == 0) return IDX_OK;
  if (!values || !scales || !aligned(values, 4)) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_quantize(x, dtype == IDX_F32, rows, row_stride, values, scales, stream));
}

int idx_quantize_rope(const void* x, int dtype, int64_t T, int H, int64_t row_stride,
                      const float* cos_table, const float* sin_table, int64_t table_rows,
                      const int64_t* positions, int rope_dim, int rope_mode, uint8_t* values,
                      uint8_t* scales, hipStream_t stream) {
  if (T < 0 || H < 1 || T > ((int64_t)1 << 40)) return IDX_ERR_ARG;
  const int64_t rows = T * H;
  int st = check_rows_input(x, dtype, rows, row_stride);
  if (st != IDX_OK) return st;
  if (rope_dim < 0 || rope_dim > IDX_HEAD_DIM || rope_dim % 16 != 0) return IDX_ERR_ARG;
  if (rope_mode != IDX_ROPE_NEOX && rope_mode != IDX_ROPE_INTERLEAVED) return IDX_ERR_ARG;
  if (table_rows < 0) return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!values || !scales || !aligned(values, 4)) return IDX_ERR_ARG;
  if (rope_dim > 0) {
    if (!cos_table || !sin_table || !aligned(cos_table, 16) || !aligned(sin_table, 16))
      return IDX_ERR_ARG;
    if (positions ? !aligned(positions, 8) : table_rows < T) return IDX_ERR_ARG;
  }
  if ((st = gate_current()) != IDX_OK) return st;
  const mxidx::RopeSpec rs{cos_table, sin_table, table_rows, positions, rope_dim,
                          rope_mode == IDX_ROPE_INTERLEAVED};
  return launched(mxidx::launch_quantize_rope(x, dtype == IDX_F32, rows, row_stride, H, rs, values,
                                              scales, stream));
}

// The checks of an idx_rope block common to the fused calls: the rotated
// prefix, the pairing, and the tables when something is rotated.
static int check_rope(const idx_rope* r) {
  if (!r) return IDX_ERR_ARG;
  if (r->rope_dim < 0 || r->rope_dim > IDX_HEAD_DIM || r->rope_dim % 16 != 0) return IDX_ERR_ARG;
  if (r->rope_mode != IDX_ROPE_NEOX && r->rope_mode != IDX_ROPE_INTERLEAVED) return IDX_ERR_ARG;
  if (r->table_rows < 0) return IDX_ERR_ARG;
  if (r->rope_dim > 0) {
    if (!r->cos_table || !r->sin_table || !aligned(r->cos_table, 16) ||
        !aligned(r->sin_table, 16))
      return IDX_ERR_ARG;
    if (r->positions && !aligned(r->positions, 8)) return IDX_ERR_ARG;
  }
  return IDX_OK;
}

static mxidx::RopeSpec rope_spec(const idx_rope* r) {
  return mxidx::RopeSpec{r->cos_table, r->sin_table, r->table_rows, r->positions, r->rope_dim,
                         r->rope_mode == IDX_ROPE_INTERLEAVED};
}

int idx_insert(const void* k, int dtype, int64_t num_tokens, int64_t k_row_stride,
               const int64_t* slot_mapping, uint8_t* cache, int64_t num_pages, int page_size,
               hipStream_t stream) {
  int st = check_rows_input(k, dtype, num_tokens, k_row_stride);
  if (st != IDX_OK) return st;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0) return IDX_ERR_ARG;
  if (num_tokens == 0) return IDX_OK;
  if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_ERR_ARG;
  if (num_pages > 0 && (!cache || !aligned(cache, 4))) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_insert(k, dtype == IDX_F32, num_tokens, k_row_stride, slot_mapping,
                                       cache, num_pages, stream));
}

int idx_insert_quantize(const void* k, int k_dtype, int64_t num_tokens, int64_t k_row_stride,
                        const int64_t* slot_mapping, uint8_t* cache, int64_t num_pages,
                        int page_size, const void* q, int q_dtype, int64_t q_rows,
                        int64_t q_row_stride, uint8_t* q_values, uint8_t* q_scales,
                        hipStream_t stream) {
  // exactly the checks of idx_insert and of idx_quantize
  int st = check_rows_input(k, k_dtype, num_tokens, k_row_stride);
  if (st != IDX_OK) return st;
  if ((st = check_rows_input(q, q_dtype, q_rows, q_row_stride)) != IDX_OK) return st;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0) return IDX_ERR_ARG;
  if (num_tokens > 0) {
    if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_ERR_ARG;
    if (num_pages > 0 && (!cache || !aligned(cache, 4))) return IDX_ERR_ARG;
  }
  if (q_rows > 0 && (!q_values || !q_scales || !aligned(q_values, 4))) return IDX_ERR_ARG;
  if (num_tokens == 0 && q_rows == 0) return IDX_OK;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_insert_quantize(k, k_dtype == IDX_F32, num_tokens, k_row_stride,
                                                slot_mapping, cache, num_pages, q,
                                                q_dtype == IDX_F32, q_rows, q_row_stride, q_values,
                                                q_scales, stream));
}

int idx_insert_quantize_rope(const void* k, int k_dtype, int64_t num_tokens,
                             int64_t k_row_stride, const int64_t* slot_mapping, uint8_t* cache,
                             int64_t num_pages, int page_size, const void* q, int q_dtype,
                             int64_t q_rows, int64_t q_row_stride, int q_heads,
                             const idx_rope* rope, uint8_t* q_values, uint8_t* q_scales,
                             hipStream_t stream) {
  int st = check_rows_input(k, k_dtype, num_tokens, k_row_stride);
  if (st != IDX_OK) return st;
  if ((st = check_rows_input(q, q_dtype, q_rows, q_row_stride)) != IDX_OK) return st;
  if ((st = check_rope(rope)) != IDX_OK) return st;
  if (q_heads < 1 || q_rows % q_heads != 0) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0) return IDX_ERR_ARG;
  if (num_tokens > 0) {
    if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_ERR_ARG;
    if (num_pages > 0 && (!cache || !aligned(cache, 4))) return IDX_ERR_ARG;
  }
  if (q_rows > 0 && (!q_values || !q_scales || !aligned(q_values, 4))) return IDX_ERR_ARG;
  // default positions (token t at table row t) need a row for every token
  if (rope->rope_dim > 0 && !rope->positions && rope->table_rows < q_rows / q_heads)
    return IDX_ERR_ARG;
  if (num_tokens == 0 && q_rows == 0) return IDX_OK;
  if ((st = gate_current()) != IDX_OK) return st;
  if (rope->rope_dim == 0)
    return launched(mxidx::launch_insert_quantize(k, k_dtype == IDX_F32, num_tokens, k_row_stride,
                                                  slot_mapping, cache, num_pages, q,
                                                  q_dtype == IDX_F32, q_rows, q_row_stride,
                                                  q_values, q_scales, stream));
  return launched(mxidx::launch_insert_quantize_rope(
      k, k_dtype == IDX_F32, num_tokens, k_row_stride, slot_mapping, cache, num_pages, q,
      q_dtype == IDX_F32, q_rows, q_row_stride, q_heads, rope_spec(rope), q_values, q_scales,
      stream));
}

int idx_gather(const uint8_t* cache, int64_t num_pages, int page_size, const int32_t* block_table,
               int64_t bt_row_stride, const int32_t* seq_lens, const int64_t* cu_seq_offsets,
               int batch, int64_t max_seq_len, int64_t total_tokens, uint8_t* k_values,
               uint8_t* k_scales, hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || batch < 0 || batch > 65535 ||
      max_seq_len < 0 || total_tokens < 0)
    return IDX_ERR_ARG;
  if (batch == 0 || max_seq_len == 0 || total_tokens == 0 || num_pages == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_seq_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq) return IDX_ERR_ARG;
  if (!cache || !aligned(cache, 16) || !block_table || !seq_lens || !cu_seq_offsets ||
      !aligned(cu_seq_offsets, 8) || !k_values || !aligned(k_values, 16) || !k_scales ||
      !aligned(k_scales, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_gather(cache, num_pages, block_table, bt_row_stride, seq_lens,
                                       cu_seq_offsets, batch, max_seq_len, total_tokens, k_values,
                                       k_scales, stream));
}

int idx_logits_prefill(const uint8_t* q_values, const uint8_t* q_scales, const uint8_t* k_values,
                       const uint8_t* k_scales, const float* weights, const int32_t* ks,
                       const int32_t* ke, int64_t T, int H, int64_t S, float* logits,
                       int64_t logits_row_stride, int clean, hipStream_t stream) {
  if (T < 0 || S < 0 || S > 0x7fffffffLL - 1024 || !heads_ok(H)) return IDX_ERR_ARG;
  if (T == 0 || S == 0) return IDX_OK;
  if (logits_row_stride < S) return IDX_ERR_ARG;
  if (!q_values || !aligned(q_values, 16) || !q_scales || !k_values || !aligned(k_values, 16) ||
      !k_scales || !aligned(k_scales, 4) || !weights || !aligned(weights, 16) || !ke || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_prefill(q_values, q_scales, k_values, k_scales, weights, ks,
                                               ke, T, H, S, logits, logits_row_stride, clean,
                                               stream));
}

int idx_logits_paged(const uint8_t* q_values, const uint8_t* q_scales, const float* weights,
                     const uint8_t* cache, int64_t num_pages, int page_size,
                     const int32_t* block_table, int64_t bt_row_stride,
                     const int32_t* context_lens, int B, int next_n, int H,
                     int64_t max_context_len, float* logits, int64_t logits_row_stride, int clean,
                     hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || B < 0 || B > IDX_MAX_DECODE_SEQS ||
      next_n < 1 || next_n > 16 || !heads_ok(H) || max_context_len < 0 ||
      max_context_len > 0x7fffffffLL - IDX_PAGE_SIZE)
    return IDX_ERR_ARG;
  if (B == 0 || max_context_len == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_context_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq || logits_row_stride < max_context_len || num_pages < 1 ||
      (int64_t)B * pages_per_seq > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (!q_values || !aligned(q_values, 16) || !q_scales || !weights || !aligned(weights, 16) ||
      !cache || !aligned(cache, 16) || !block_table || !context_lens || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_paged(q_values, q_scales, weights, cache, num_pages,
                                             block_table, bt_row_stride, context_lens, B, next_n,
                                             H, max_context_len, logits, logits_row_stride, clean,
                                             stream));
}

int idx_logits_paged_insert(const void* q, const void* k_new, int dtype, const float* weights,
                            uint8_t* cache, int64_t num_pages, int page_size,
                            const int32_t* block_table, int64_t bt_row_stride,
                            const int32_t* context_lens, int B, int next_n, int H,
                            int64_t max_context_len, float* logits, int64_t logits_row_stride,
                            int clean, hipStream_t stream) {
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || B < 0 || B > IDX_MAX_DECODE_SEQS ||
      next_n < 1 || next_n > 16 || !heads_ok(H) || max_context_len < 0 ||
      max_context_len > 0x7fffffffLL - IDX_PAGE_SIZE)
    return IDX_ERR_ARG;
  if (B == 0 || max_context_len == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_context_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq || logits_row_stride < max_context_len || num_pages < 1 ||
      (int64_t)B * pages_per_seq > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (!q || !aligned(q, 16) || !k_new || !aligned(k_new, 16) || !weights || !aligned(weights, 16) ||
      !cache || !aligned(cache, 16) || !block_table || !context_lens || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_paged_insert(
      q, k_new, dtype == IDX_F32, weights, cache, num_pages, block_table, bt_row_stride,
      context_lens, B, next_n, H, max_context_len, logits, logits_row_stride, clean, stream));
}

int idx_logits_paged_insert_rope(const void* q, const void* k_new, int dtype,
                                 const float* weights, uint8_t* cache, int64_t num_pages,
                                 int page_size, const int32_t* block_table, int64_t bt_row_stride,
                                 const int32_t* context_lens, int B, int next_n, int H,
                                 int64_t max_context_len, float* logits,
                                 int64_t logits_row_stride, int clean, const idx_rope* rope,
                                 hipStream_t stream) {
  int st = check_rope(rope);
  if (st != IDX_OK) return st;
  // the in-wave rotation takes neox partners from one other lane block
  if (rope->rope_mode == IDX_ROPE_NEOX && rope->rope_dim != 0 && rope->rope_dim != 64 &&
      rope->rope_dim != 128)
    return IDX_ERR_ARG;
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || B < 0 || B > IDX_MAX_DECODE_SEQS ||
      next_n < 1 || next_n > 16 || !heads_ok(H) || max_context_len < 0 ||
      max_context_len > 0x7fffffffLL - IDX_PAGE_SIZE)
    return IDX_ERR_ARG;
  if (B == 0 || max_context_len == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_context_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq || logits_row_stride < max_context_len || num_pages < 1 ||
      (int64_t)B * pages_per_seq > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (!q || !aligned(q, 16) || !k_new || !aligned(k_new, 16) || !weights || !aligned(weights, 16) ||
      !cache || !aligned(cache, 16) || !block_table || !context_lens || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_logits_paged_insert_rope(
      q, k_new, dtype == IDX_F32, weights, cache, num_pages, block_table, bt_row_stride,
      context_lens, B, next_n, H, max_context_len, logits, logits_row_stride, clean,
      rope_spec(rope), stream));
}

int idx_topk_merge(const float* values, const int32_t* indices, int world, int64_t rows, int k_in,
                   int interleave, int k, int32_t* out_idx, hipStream_t stream) {
  if (world < 1 || rows < 0 || k_in < 1 || interleave < 1 || k < 1 || k > IDX_TOPK_MAX ||
      (int64_t)world * k_in > IDX_MERGE_MAX_CANDIDATES || rows > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!values || !aligned(values, 4) || !indices || !aligned(indices, 4) || !out_idx) return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_topk_merge(values, indices, world, k_in, rows, interleave, k,
                                           out_idx, stream));
}

int idx_topk(const float* logits, int64_t rows, int64_t logits_row_stride, const int32_t* ks,
             const int32_t* ke, int k, int32_t* out_idx, hipStream_t stream) {
  if (rows < 0 || k < 1 || k > IDX_TOPK_MAX || logits_row_stride < 0 ||
      rows > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!logits || !aligned(logits, 4) || !ke || !out_idx) return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_topk(logits, rows, logits_row_stride, ks, ke, k, out_idx, stream));
}

size_t idx_topk_workspace_bytes(int64_t rows, int64_t logits_row_stride) {
  if (rows < 0 || logits_row_stride < 0 || rows > 0x7fffffffLL) return 0;
  return (size_t)mxidx::topk_workspace_bytes(rows, logits_row_stride);
}

int idx_topk_ws(const float* logits, int64_t rows, int64_t logits_row_stride, const int32_t* ks,
                const int32_t* ke, int k, int32_t* out_idx, void* workspace,
                size_t workspace_bytes, hipStream_t stream) {
  if (rows < 0 || k < 1 || k > IDX_TOPK_MAX || logits_row_stride < 0 ||
      rows > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!logits || !aligned(logits, 4) || !ke || !out_idx) return IDX_ERR_ARG;
  const size_t need = idx_topk_workspace_bytes(rows, logits_row_stride);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_topk_ws(logits, rows, logits_row_stride, ks, ke, k, out_idx,
                                        workspace, stream));
}

int idx_quantize_fp8(const void* x, int dtype, int64_t rows, int64_t row_stride, int scale_fmt,
                     uint8_t* values, float* scales, const float* w_in, float* w_out,
                     hipStream_t stream) {
  int st = check_rows_input(x, dtype, rows, row_stride);
  if (st != IDX_OK) return st;
  if (scale_fmt != IDX_FP8_SCALE_F32 && scale_fmt != IDX_FP8_SCALE_POW2) return IDX_ERR_ARG;
  if ((w_in == nullptr) != (w_out == nullptr)) return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!values || !aligned(values, 16) || !scales || !aligned(scales, 4)) return IDX_ERR_ARG;
  if (w_in && (!aligned(w_in, 4) || !aligned(w_out, 4))) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_quantize_fp8(x, dtype == IDX_F32, rows, row_stride,
                                             scale_fmt == IDX_FP8_SCALE_POW2, values, scales, w_in,
                                             w_out, stream));
}

int idx_insert_fp8(const void* k, int dtype, int64_t num_tokens, int64_t k_row_stride,
                   int scale_fmt, const int64_t* slot_mapping, uint8_t* cache, int64_t num_pages,
                   int page_size, hipStream_t stream) {
  int st = check_rows_input(k, dtype, num_tokens, k_row_stride);
  if (st != IDX_OK) return st;
  if (scale_fmt != IDX_FP8_SCALE_F32 && scale_fmt != IDX_FP8_SCALE_POW2) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0) return IDX_ERR_ARG;
  if (num_tokens == 0) return IDX_OK;
  if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_ERR_ARG;
  if (num_pages > 0 && (!cache || !aligned(cache, 16))) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_insert_fp8(k, dtype == IDX_F32, num_tokens, k_row_stride,
                                           scale_fmt == IDX_FP8_SCALE_POW2, slot_mapping, cache,
                                           num_pages, stream));
}

int idx_gather_fp8(const uint8_t* cache, int64_t num_pages, int page_size,
                   const int32_t* block_table, int64_t bt_row_stride, const int32_t* seq_lens,
                   const int64_t* cu_seq_offsets, int batch, int64_t max_seq_len,
                   int64_t total_tokens, uint8_t* k_values, float* k_scales, hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || batch < 0 || batch > 65535 ||
      max_seq_len < 0 || total_tokens < 0)
    return IDX_ERR_ARG;
  if (batch == 0 || max_seq_len == 0 || total_tokens == 0 || num_pages == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_seq_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq) return IDX_ERR_ARG;
  if (!cache || !aligned(cache, 16) || !block_table || !seq_lens || !cu_seq_offsets ||
      !aligned(cu_seq_offsets, 8) || !k_values || !aligned(k_values, 16) || !k_scales ||
      !aligned(k_scales, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_gather_fp8(cache, num_pages, block_table, bt_row_stride, seq_lens,
                                           cu_seq_offsets, batch, max_seq_len, total_tokens,
                                           k_values, k_scales, stream));
}

int idx_logits_prefill_fp8(const uint8_t* q_values, const float* weights, const uint8_t* k_values,
                           const float* k_scales, const int32_t* ks, const int32_t* ke, int64_t T,
                           int H, int64_t S, float* logits, int64_t logits_row_stride, int clean,
                           hipStream_t stream) {
  if (T < 0 || S < 0 || S > 0x7fffffffLL - 1024 || !heads_ok(H)) return IDX_ERR_ARG;
  if (T == 0 || S == 0) return IDX_OK;
  if (logits_row_stride < S) return IDX_ERR_ARG;
  if (!q_values || !aligned(q_values, 16) || !weights || !aligned(weights, 16) || !k_values ||
      !aligned(k_values, 16) || !k_scales || !aligned(k_scales, 4) || !ke || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_prefill_fp8(q_values, weights, k_values, k_scales, ks, ke, T,
                                                   H, S, logits, logits_row_stride, clean, stream));
}

int idx_logits_paged_fp8(const uint8_t* q_values, const float* weights, const uint8_t* cache,
                         int64_t num_pages, int page_size, const int32_t* block_table,
                         int64_t bt_row_stride, const int32_t* context_lens, int B, int next_n,
                         int H, int64_t max_context_len, float* logits, int64_t logits_row_stride,
                         int clean, hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || B < 0 || B > IDX_MAX_DECODE_SEQS ||
      next_n < 1 || next_n > 16 || !heads_ok(H) || max_context_len < 0 ||
      max_context_len > 0x7fffffffLL - IDX_PAGE_SIZE)
    return IDX_ERR_ARG;
  if (B == 0 || max_context_len == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_context_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq || logits_row_stride < max_context_len || num_pages < 1 ||
      (int64_t)B * pages_per_seq > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (!q_values || !aligned(q_values, 16) || !weights || !aligned(weights, 16) || !cache ||
      !aligned(cache, 16) || !block_table || !context_lens || !logits || !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_paged_fp8(q_values, weights, cache, num_pages, block_table,
                                                 bt_row_stride, context_lens, B, next_n, H,
                                                 max_context_len, logits, logits_row_stride, clean,
                                                 stream));
}

int idx_logits_paged_insert_fp8(const void* q, const void* k_new, int dtype, const float* weights,
                                int scale_fmt, uint8_t* cache, int64_t num_pages, int page_size,
                                const int32_t* block_table, int64_t bt_row_stride,
                                const int32_t* context_lens, int B, int next_n, int H,
                                int64_t max_context_len, float* logits,
                                int64_t logits_row_stride, int clean, hipStream_t stream) {
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (scale_fmt != IDX_FP8_SCALE_F32 && scale_fmt != IDX_FP8_SCALE_POW2) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0 || B < 0 || B > IDX_MAX_DECODE_SEQS ||
      next_n < 1 || next_n > 16 || !heads_ok(H) || max_context_len < 0 ||
      max_context_len > 0x7fffffffLL - IDX_PAGE_SIZE)
    return IDX_ERR_ARG;
  if (B == 0 || max_context_len == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_context_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq || logits_row_stride < max_context_len || num_pages < 1 ||
      (int64_t)B * pages_per_seq > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (!q || !aligned(q, 16) || !k_new || !aligned(k_new, 16) || !weights || !aligned(weights, 16) ||
      !cache || !aligned(cache, 16) || !block_table || !context_lens || !logits ||
      !aligned(logits, 4))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_logits_paged_insert_fp8(
      q, k_new, dtype == IDX_F32, weights, scale_fmt == IDX_FP8_SCALE_POW2, cache, num_pages,
      block_table, bt_row_stride, context_lens, B, next_n, H, max_context_len, logits,
      logits_row_stride, clean, stream));
}

int idx_kpool_insert(const void* k, int dtype, int64_t n, int64_t k_row_stride,
                     const float* gate_score, const float* ape, const int64_t* slot_mapping,
                     int kpool, int cache_format, int fp8_scale_fmt, uint8_t* cache,
                     int64_t num_pages, int page_size, float* compressed, hipStream_t stream) {
  int st = check_rows_input(k, dtype, n, k_row_stride);
  if (st != IDX_OK) return st;
  if (kpool < 1 || kpool > IDX_KPOOL_MAX) return IDX_ERR_ARG;
  if (cache_format != IDX_CACHE_MXFP4 && cache_format != IDX_CACHE_FP8) return IDX_ERR_ARG;
  if (fp8_scale_fmt != IDX_FP8_SCALE_F32 && fp8_scale_fmt != IDX_FP8_SCALE_POW2) return IDX_ERR_ARG;
  if (page_size != IDX_PAGE_SIZE || num_pages < 0) return IDX_ERR_ARG;
  if (n < kpool) return IDX_OK;                 // no pool completes
  if (!gate_score || !aligned(gate_score, 16) || !ape || !aligned(ape, 16) || !slot_mapping ||
      !aligned(slot_mapping, 8))
    return IDX_ERR_ARG;
  if (compressed && !aligned(compressed, 16)) return IDX_ERR_ARG;
  if (num_pages > 0 && (!cache || !aligned(cache, 16))) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_kpool_insert(k, dtype == IDX_F32, n, k_row_stride, gate_score, ape,
                                             slot_mapping, kpool, cache_format == IDX_CACHE_FP8,
                                             fp8_scale_fmt == IDX_FP8_SCALE_POW2, cache, num_pages,
                                             compressed, stream));
}

int idx_topk_noalloc(const float* logits, int64_t rows, int64_t logits_row_stride,
                     const int32_t* ks, const int32_t* ke, int k, int32_t* out_idx,
                     hipStream_t stream) {
  if (rows < 0 || k < 1 || k > IDX_TOPK_MAX || logits_row_stride < 0 || rows > 0x7fffffffLL)
    return IDX_ERR_ARG;
  if (rows == 0) return IDX_OK;
  if (!logits || !aligned(logits, 4) || !ke || !out_idx) return IDX_ERR_ARG;
  // the library's scratch holds at most IDX_TOPK_NOALLOC_MAX_WORKSPACE bytes
  if (idx_topk_workspace_bytes(rows, logits_row_stride) > (size_t)IDX_TOPK_NOALLOC_MAX_WORKSPACE)
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_topk_noalloc(logits, rows, logits_row_stride, ks, ke, k, out_idx,
                                             stream));
}

int idx_step_map(const int32_t* seq_lens, const int32_t* query_lens, int B, int32_t* block_table,
                 int64_t bt_row_stride, int64_t bt_pages, const int32_t* free_pages,
                 int64_t num_free, const int64_t* free_start, int64_t* free_next, int page_size,
                 int columns, int64_t num_rows, int64_t* slot_mapping, int64_t* positions,
                 int32_t* row_seq, int32_t* ks, int32_t* ke, int64_t* cu_seq_offsets,
                 hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || B < 0 || B > IDX_MAX_DECODE_SEQS || num_rows < 0 ||
      num_rows > 0x7fffffffLL || num_free < 0 || bt_pages < 0 || bt_row_stride < bt_pages)
    return IDX_ERR_ARG;
  if (columns != IDX_COLUMNS_SEQUENCE && columns != IDX_COLUMNS_GATHERED) return IDX_ERR_ARG;
  if (B > 0) {
    if (!seq_lens || !aligned(seq_lens, 4) || !query_lens || !aligned(query_lens, 4))
      return IDX_ERR_ARG;
    if (slot_mapping && bt_pages > 0 && !block_table) return IDX_ERR_ARG;
  }
  // a list of no pages is still a list: its pages are all lacking
  if (free_pages ? !free_start || !aligned(free_start, 8) : num_free > 0) return IDX_ERR_ARG;
  if (free_next && (!aligned(free_next, 8) || free_next == free_start)) return IDX_ERR_ARG;
  if (!aligned(block_table, 4) || !aligned(free_pages, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 8) || !aligned(row_seq, 4) || !aligned(ks, 4) || !aligned(ke, 4) ||
      !aligned(cu_seq_offsets, 8))
    return IDX_ERR_ARG;
  if (num_rows == 0 && !free_next && !cu_seq_offsets) return IDX_OK;
  int st = gate_current();
  if (st != IDX_OK) return st;
  const mxidx::StepMapArgs a{seq_lens,   query_lens, B,         columns == IDX_COLUMNS_GATHERED,
                             block_table, bt_row_stride, bt_pages, free_pages, num_free, free_start,
                             free_next,  num_rows,   slot_mapping, positions, row_seq, ks, ke,
                             cu_seq_offsets};
  return launched(mxidx::launch_step_map(a, stream));
}

// `count` rows of `width` values: a stride that steps over whole, aligned rows.
static bool stride_ok(int64_t stride, int64_t count, int width, int align) {
  return count <= 1 || (stride >= width && stride % align == 0);
}

static int check_heads(const idx_heads* s, int dtype, int64_t T) {
  if (s->heads < 0 || s->norm < IDX_NORM_NONE || s->norm > IDX_NORM_LAYER) return IDX_ERR_ARG;
  if (s->heads == 0 || T == 0) return IDX_OK;
  const int al = dtype == IDX_BF16 ? 8 : 4;
  if (!s->x || !aligned(s->x, 16) || !s->out || !aligned(s->out, 16)) return IDX_ERR_ARG;
  if (!stride_ok(s->row_stride, T, IDX_HEAD_DIM, al) ||
      !stride_ok(s->head_stride, s->heads, IDX_HEAD_DIM, al) ||
      !stride_ok(s->out_row_stride, T, IDX_HEAD_DIM, al) ||
      !stride_ok(s->out_head_stride, s->heads, IDX_HEAD_DIM, al))
    return IDX_ERR_ARG;
  // in place: row by row
  if (s->out == s->x && ((T > 1 && s->out_row_stride != s->row_stride) ||
                         (s->heads > 1 && s->out_head_stride != s->head_stride)))
    return IDX_ERR_ARG;
  if (s->norm != IDX_NORM_NONE &&
      (!aligned(s->weight, 16) || !aligned(s->bias, 16) || !(s->eps >= 0.f)))
    return IDX_ERR_ARG;
  return IDX_OK;
}

static mxidx::HeadsSpec heads_spec(const idx_heads* s) {
  if (!s) return mxidx::HeadsSpec{};
  const bool on = s->norm != IDX_NORM_NONE;
  return mxidx::HeadsSpec{s->x,     s->out,  s->row_stride, s->head_stride, s->out_row_stride,
                          s->out_head_stride, s->heads, s->norm, on ? s->weight : nullptr,
                          on ? s->bias : nullptr, s->eps};
}

int idx_norm_rope(const idx_heads* q, const idx_heads* k, int dtype, int64_t T,
                  const idx_rope* rope, hipStream_t stream) {
  int st = check_rope(rope);
  if (st != IDX_OK) return st;
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (T < 0 || T > ((int64_t)1 << 40)) return IDX_ERR_ARG;
  if (q && (st = check_heads(q, dtype, T)) != IDX_OK) return st;
  if (k && (st = check_heads(k, dtype, T)) != IDX_OK) return st;
  const int64_t heads = (int64_t)(q ? q->heads : 0) + (k ? k->heads : 0);
  if (heads > (1 << 20)) return IDX_ERR_ARG;
  if (T == 0 || heads == 0) return IDX_OK;
  if (T > ((int64_t)1 << 27) / heads) return IDX_ERR_ARG;   // the grid: 16 lanes a row
  if (rope->rope_dim > 0 && !rope->positions && rope->table_rows < T) return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  return launched(mxidx::launch_norm_rope(heads_spec(q), heads_spec(k), dtype == IDX_F32, T,
                                          rope_spec(rope), stream));
}

static bool latent_ok(int latent) { return latent == 128 || latent == 256 || latent == 512; }

// idx_latent_insert and idx_latent_insert_mxfp4 (mx).
static int latent_insert(const void* kv, int dtype, int64_t T, int64_t kv_row_stride, int latent,
                         int norm, const float* weight, double eps, const idx_rope* rope,
                         const int64_t* slot_mapping, void* cache, int64_t num_pages, int page_size,
                         const void* q_pe, int H, int64_t q_row_stride, int64_t q_head_stride,
                         void* q_out, int64_t out_row_stride, int64_t out_head_stride, bool mx,
                         hipStream_t stream) {
  int st = check_rope(rope);
  if (st != IDX_OK) return st;
  if (rope->rope_dim != IDX_LATENT_ROPE) return IDX_ERR_ARG;
  if (dtype != IDX_BF16 && dtype != IDX_F32) return IDX_ERR_ARG;
  if (!latent_ok(latent) || page_size != IDX_PAGE_SIZE || num_pages < 0 ||
      num_pages > ((int64_t)1 << 40) || T < 0 || H < 0)
    return IDX_ERR_ARG;
  // the grid is a wave a token and 8 lanes a query row, and a launch has fewer than 2^32 lanes
  if (T > (1 << 24) || (q_pe && T * H > ((int64_t)1 << 28))) return IDX_ERR_ARG;
  if (norm != IDX_NORM_NONE && norm != IDX_NORM_RMS) return IDX_ERR_ARG;
  if (T == 0) return IDX_OK;
  const int al = dtype == IDX_BF16 ? 8 : 4;
  if (!kv || !aligned(kv, 16) || !stride_ok(kv_row_stride, T, latent + IDX_LATENT_ROPE, al))
    return IDX_ERR_ARG;
  if (norm == IDX_NORM_RMS && (!aligned(weight, 16) || !(eps >= 0.0))) return IDX_ERR_ARG;
  if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_ERR_ARG;
  if (num_pages > 0 && (!cache || !aligned(cache, 16))) return IDX_ERR_ARG;
  if (!rope->positions && rope->table_rows < T) return IDX_ERR_ARG;
  const bool has_q = q_pe && H > 0;
  if (has_q && (!aligned(q_pe, 16) || !q_out || !aligned(q_out, 16) ||
                !stride_ok(q_row_stride, T, IDX_LATENT_ROPE, al) ||
                !stride_ok(q_head_stride, H, IDX_LATENT_ROPE, al) ||
                !stride_ok(out_row_stride, T, IDX_LATENT_ROPE, 8) ||
                !stride_ok(out_head_stride, H, IDX_LATENT_ROPE, 8)))
    return IDX_ERR_ARG;
  if (has_q && q_out == q_pe &&                // in place: row by row
      (dtype != IDX_BF16 || (T > 1 && out_row_stride != q_row_stride) ||
       (H > 1 && out_head_stride != q_head_stride)))
    return IDX_ERR_ARG;
  if ((st = gate_current()) != IDX_OK) return st;
  const mxidx::LatentSpec a{kv, T, kv_row_stride, norm, norm == IDX_NORM_RMS ? weight : nullptr,
                            eps, slot_mapping, cache, num_pages * IDX_PAGE_SIZE,
                            has_q ? q_pe : nullptr, H, q_row_stride, q_head_stride, q_out,
                            out_row_stride, out_head_stride};
  return launched(mxidx::launch_latent_insert(a, dtype == IDX_F32, latent, mx, rope_spec(rope), stream));
}

int idx_latent_insert(const void* kv, int dtype, int64_t T, int64_t kv_row_stride, int latent,
                      int norm, const float* weight, float eps, const idx_rope* rope,
                      const int64_t* slot_mapping, void* cache, int64_t num_pages, int page_size,
                      const void* q_pe, int H, int64_t q_row_stride, int64_t q_head_stride,
                      void* q_out, int64_t out_row_stride, int64_t out_head_stride,
                      hipStream_t stream) {
  return latent_insert(kv, dtype, T, kv_row_stride, latent, norm, weight, eps, rope, slot_mapping, cache,
                       num_pages, page_size, q_pe, H, q_row_stride, q_head_stride, q_out, out_row_stride,
                       out_head_stride, false, stream);
}

int idx_latent_insert_mxfp4(const void* kv, int dtype, int64_t T, int64_t kv_row_stride, int latent,
                            int norm, const float* weight, double eps, const idx_rope* rope,
                            const int64_t* slot_mapping, uint8_t* cache, int64_t num_pages, int page_size,
                            const void* q_pe, int H, int64_t q_row_stride, int64_t q_head_stride,
                            void* q_out, int64_t out_row_stride, int64_t out_head_stride,
                            hipStream_t stream) {
  return latent_insert(kv, dtype, T, kv_row_stride, latent, norm, weight, eps, rope, slot_mapping, cache,
                       num_pages, page_size, q_pe, H, q_row_stride, q_head_stride, q_out, out_row_stride,
                       out_head_stride, true, stream);
}

int idx_latent_gather_mxfp4(const uint8_t* cache, int64_t num_pages, int page_size, int latent,
                            const int32_t* block_table, int64_t bt_row_stride, const int32_t* seq_lens,
                            const int64_t* cu_seq_offsets, int batch, int64_t max_seq_len,
                            int64_t total_tokens, void* out, int64_t out_row_stride, hipStream_t stream) {
  if (page_size != IDX_PAGE_SIZE || !latent_ok(latent) || num_pages < 0 || num_pages > ((int64_t)1 << 40) ||
      batch < 0 || batch > IDX_MAX_DECODE_SEQS || max_seq_len < 0 || max_seq_len > IDX_GATHER_MAX_TOKENS ||
      total_tokens < 0)
    return IDX_ERR_ARG;
  if (batch == 0 || max_seq_len == 0 || total_tokens == 0 || num_pages == 0) return IDX_OK;
  const int64_t pages_per_seq = (max_seq_len + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq) return IDX_ERR_ARG;
  if (!cache || !aligned(cache, 16) || !block_table || !aligned(block_table, 4) || !seq_lens ||
      !aligned(seq_lens, 4) || !cu_seq_offsets || !aligned(cu_seq_offsets, 8) || !out || !aligned(out, 16) ||
      !stride_ok(out_row_stride, total_tokens, latent + IDX_LATENT_ROPE, 8))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  return launched(mxidx::launch_latent_gather(
      {cache, num_pages, block_table, bt_row_stride, seq_lens, cu_seq_offsets, batch, max_seq_len,
       total_tokens, out, out_row_stride},
      latent, stream));
}

// What the two calls below share: sizes that the kernels' grid and indexes take.  A row takes
// two workgroups of 256 lanes at most where rows are many, and a launch has fewer than 2^32.
static bool attn_sizes_ok(int64_t rows, int H, int latent, int64_t max_tokens) {
  return rows >= 0 && H >= 1 && H <= IDX_MAX_HEADS && rows <= IDX_ATTN_MAX_ROWS &&
         latent_ok(latent) && max_tokens >= 0 && max_tokens <= IDX_ATTN_MAX_TOKENS;
}

size_t idx_attn_workspace_bytes(int64_t rows, int H, int latent, int64_t entries) {
  if (!attn_sizes_ok(rows, H, latent, entries)) return 0;
  return (size_t)mxidx::attn_workspace_bytes(rows, H, latent, entries, false);
}

size_t idx_attn_workspace_bytes_mxfp4(int64_t rows, int H, int latent, int64_t entries) {
  if (!attn_sizes_ok(rows, H, latent, entries)) return 0;
  return (size_t)mxidx::attn_workspace_bytes(rows, H, latent, entries, true);
}

size_t idx_attn_workspace_max_bytes(int64_t rows, int H, int latent, int64_t entries) {
  if (!attn_sizes_ok(rows, H, latent, entries)) return 0;
  return (size_t)mxidx::attn_workspace_max_bytes(rows, H, latent, entries);
}

// idx_attn_paged and idx_attn_paged_mxfp4 (mx).
static int attn_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t rows, int H,
                      int latent, const void* cache, int64_t num_pages, int page_size,
                      const int32_t* block_table, int64_t bt_row_stride, int B,
                      const int32_t* row_seq, const int32_t* ks, const int32_t* ke,
                      const int32_t* indices, int64_t idx_row_stride, int k, int64_t max_tokens,
                      float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                      float* lse, void* workspace, size_t workspace_bytes, bool mx,
                      hipStream_t stream) {
  if (!attn_sizes_ok(rows, H, latent, max_tokens) || page_size != IDX_PAGE_SIZE || num_pages < 0 ||
      num_pages > IDX_ATTN_MAX_PAGES || B < 0)
    return IDX_ERR_ARG;
  if (rows == 0 || B == 0) return IDX_OK;     // no row belongs to a sequence
  const int64_t pages_per_seq = (max_tokens + IDX_PAGE_SIZE - 1) / IDX_PAGE_SIZE;
  if (bt_row_stride < pages_per_seq) return IDX_ERR_ARG;
  if (!row_seq && rows % B != 0) return IDX_ERR_ARG;
  if (!q || !aligned(q, 16) || !stride_ok(q_row_stride, rows, latent + IDX_LATENT_ROPE, 8) ||
      !stride_ok(q_head_stride, H, latent + IDX_LATENT_ROPE, 8))
    return IDX_ERR_ARG;
  if (!out || !aligned(out, 8) || !stride_ok(out_row_stride, rows, latent, 4) ||
      !stride_ok(out_head_stride, H, latent, 4))
    return IDX_ERR_ARG;
  if (!ke || !aligned(ke, 4) || !aligned(ks, 4) || !aligned(row_seq, 4) || !aligned(lse, 4))
    return IDX_ERR_ARG;
  if (indices && (k < 0 || k > IDX_ATTN_MAX_TOKENS || !aligned(indices, 4) || !stride_ok(idx_row_stride, rows, k, 1)))
    return IDX_ERR_ARG;
  if (max_tokens > 0 && (!block_table || !aligned(block_table, 4))) return IDX_ERR_ARG;
  if (num_pages > 0 && (!cache || !aligned(cache, 16))) return IDX_ERR_ARG;
  const int64_t entries = indices ? k : max_tokens;
  const size_t need = mx ? idx_attn_workspace_bytes_mxfp4(rows, H, latent, entries)
                         : idx_attn_workspace_bytes(rows, H, latent, entries);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  const mxidx::AttnArgs a{q, q_row_stride, q_head_stride, rows, H, cache, num_pages, block_table,
                          bt_row_stride, B, row_seq, row_seq ? 1 : rows / B, ks, ke, indices,
                          idx_row_stride, k, max_tokens, scale, out, out_row_stride,
                          out_head_stride, lse};
  return launched(mxidx::launch_attn_paged(a, latent, mx, workspace, stream));
}

int idx_attn_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t rows, int H,
                   int latent, const void* cache, int64_t num_pages, int page_size,
                   const int32_t* block_table, int64_t bt_row_stride, int B,
                   const int32_t* row_seq, const int32_t* ks, const int32_t* ke,
                   const int32_t* indices, int64_t idx_row_stride, int k, int64_t max_tokens,
                   float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                   float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return attn_paged(q, q_row_stride, q_head_stride, rows, H, latent, cache, num_pages, page_size, block_table,
                    bt_row_stride, B, row_seq, ks, ke, indices, idx_row_stride, k, max_tokens, scale, out,
                    out_row_stride, out_head_stride, lse, workspace, workspace_bytes, false, stream);
}

int idx_attn_paged_mxfp4(const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t rows, int H,
                         int latent, const uint8_t* cache, int64_t num_pages, int page_size,
                         const int32_t* block_table, int64_t bt_row_stride, int B,
                         const int32_t* row_seq, const int32_t* ks, const int32_t* ke,
                         const int32_t* indices, int64_t idx_row_stride, int k, int64_t max_tokens,
                         float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                         float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return attn_paged(q, q_row_stride, q_head_stride, rows, H, latent, cache, num_pages, page_size, block_table,
                    bt_row_stride, B, row_seq, ks, ke, indices, idx_row_stride, k, max_tokens, scale, out,
                    out_row_stride, out_head_stride, lse, workspace, workspace_bytes, true, stream);
}

// Sizes that the kernel's grid and indexes take; T and B above 0.
static bool prompt_sizes_ok(int64_t T, int Hq, int Hk, int dk, int dv, int64_t S, int B, int64_t max_seq_len) {
  const bool dims = (dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128);
  if (!dims || T < 0 || T > IDX_ATTN_MAX_ROWS || Hq < 1 || Hq > IDX_PROMPT_MAX_HEADS || Hk < 1 || Hq % Hk != 0 || S < 0 ||
      S > ((int64_t)1 << 40) || B < 0 || B > IDX_PROMPT_MAX_SEQS || max_seq_len < 0 || max_seq_len > IDX_ATTN_MAX_TOKENS)
    return false;
  return T == 0 || B == 0 || mxidx::prompt_lanes(T, Hq, Hk, B, max_seq_len) < ((int64_t)1 << 32);
}

size_t idx_attn_prompt_workspace_bytes(int64_t T, int Hq, int Hk, int dk, int dv, int B, int64_t max_seq_len) {
  if (!prompt_sizes_ok(T, Hq, Hk, dk, dv, 0, B, max_seq_len)) return 0;
  return (size_t)mxidx::prompt_workspace_bytes(T, Hq, Hk, dv, B, max_seq_len);
}

int idx_attn_prompt(const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T, int Hq, const void* k,
                    int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                    int64_t v_head_stride, int64_t S, int Hk, int dk, int dv, const int32_t* seq_lens,
                    const int32_t* query_lens, int B, int64_t max_seq_len, int causal, float scale, void* out,
                    int64_t out_row_stride, int64_t out_head_stride, float* lse, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  if (!prompt_sizes_ok(T, Hq, Hk, dk, dv, S, B, max_seq_len)) return IDX_ERR_ARG;
  if (T == 0 || B == 0) return IDX_OK;        // no row belongs to a request
  if (!q || !aligned(q, 16) || !stride_ok(q_row_stride, T, dk, 8) || !stride_ok(q_head_stride, Hq, dk, 8))
    return IDX_ERR_ARG;
  // a tile's rows are addressed in 32 bits from its first
  if (S > 0 && (!k || !aligned(k, 16) || !stride_ok(k_row_stride, S, dk, 8) || !stride_ok(k_head_stride, Hk, dk, 8) ||
                !v || !aligned(v, 16) || !stride_ok(v_row_stride, S, dv, 8) || !stride_ok(v_head_stride, Hk, dv, 8) ||
                (S > 1 && (k_row_stride > IDX_PROMPT_MAX_STRIDE || v_row_stride > IDX_PROMPT_MAX_STRIDE))))
    return IDX_ERR_ARG;
  if (!out || !aligned(out, 8) || !stride_ok(out_row_stride, T, dv, 4) || !stride_ok(out_head_stride, Hq, dv, 4))
    return IDX_ERR_ARG;
  if (!seq_lens || !aligned(seq_lens, 4) || !query_lens || !aligned(query_lens, 4) || !aligned(lse, 4))
    return IDX_ERR_ARG;
  const size_t need = idx_attn_prompt_workspace_bytes(T, Hq, Hk, dk, dv, B, max_seq_len);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return IDX_ERR_ARG;
  int st = gate_current();
  if (st != IDX_OK) return st;
  const mxidx::PromptArgs a{q, q_row_stride, q_head_stride, T, Hq, k, S > 1 ? k_row_stride : dk, k_head_stride,
                            v, S > 1 ? v_row_stride : dv, v_head_stride, S, Hk, seq_lens, query_lens, B, max_seq_len,
                            causal != 0, scale, out, out_row_stride, out_head_stride, lse};
  return launched(mxidx::launch_attn_prompt(a, dk, dv, workspace, stream));
}

}  // extern "C"

namespace {

// An argument of a call out of its 8-byte word; false: it does not fit.
template <class T>
bool from_word(int64_t word, T& x) {
  if constexpr (std::is_pointer_v<T>) {
    x = reinterpret_cast<T>(word);
  } else if constexpr (std::is_floating_point_v<T>) {
    double d;
    std::memcpy(&d, &word, 8);
    x = (T)d;
  } else {
    x = (T)word;
    // a size has no sign, and nothing fits it twice
    return (int64_t)x == word && (std::is_signed_v<T> || word >= 0);
  }
  return true;
}

template <class... A, size_t... i>
int apply(int (*call)(A...), const char* words, std::index_sequence<i...>) {
  std::tuple<A...> args;
  const auto word = [&](size_t k) {
    int64_t w;
    std::memcpy(&w, words + 8 * k, 8);
    return w;
  };
  if (!(from_word(word(i), std::get<i>(args)) && ...)) return IDX_ERR_ARG;
  return call(std::get<i>(args)...);
}

template <auto call>
struct Entry;
template <class... A, int (*call)(A...)>
struct Entry<call> {
  static constexpr int kCount = sizeof...(A);
  static int run(const char* words) { return apply(call, words, std::make_index_sequence<sizeof...(A)>()); }
};

struct EntryRow {
  const char* name;
  int count;
  int (*run)(const char*);
};
#define MXIDX_ENTRY(f) {#f, Entry<f>::kCount, Entry<f>::run}
const EntryRow kEntries[] = {
    MXIDX_ENTRY(idx_step_map),        MXIDX_ENTRY(idx_norm_rope),
    MXIDX_ENTRY(idx_latent_insert),   MXIDX_ENTRY(idx_latent_insert_mxfp4),
    MXIDX_ENTRY(idx_latent_gather_mxfp4), MXIDX_ENTRY(idx_attn_paged),
    MXIDX_ENTRY(idx_attn_paged_mxfp4), MXIDX_ENTRY(idx_attn_prompt),
};
#undef MXIDX_ENTRY
constexpr int kEntryCount = sizeof(kEntries) / sizeof(kEntries[0]);

}  // namespace

extern "C" {

int idx_entry(const char* name) {
  for (int i = 0; name && i < kEntryCount; ++i)
    if (std::strcmp(name, kEntries[i].name) == 0) return i;
  return -1;
}

int idx_call(int entry, const void* words, int count) {
  if (entry < 0 || entry >= kEntryCount || !words || count != kEntries[entry].count) return IDX_ERR_ARG;
  return kEntries[entry].run(static_cast<const char*>(words));
}

}  // extern "C"
