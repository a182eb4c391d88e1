// Launch interface of the kernels over the one-kind paged caches (BF16 pages
// and 4-bit pages): position-rotated appends, the 4-bit read-back and the
// windowed attention.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace oscar {

constexpr int kTile4 = 16;                     // tokens of a 4-bit tile
constexpr int kTile4Bytes = 2176;              // K codes | V codes | K scales | V scales
constexpr int kTile4V = 1024, kTile4Scales = 2048;
constexpr int kBlock4Bytes = 4 * kTile4Bytes;  // one page of one KV head

// The page table part of a view.
struct PageRefs {
  const int32_t* table = nullptr;  // [batch][max_pages]
  int64_t num_pages = 0;
  int32_t max_pages = 0, batch = 0;
};

// The tokens of a call: request b owns [cu[b], cu[b + 1]), or token b alone without cu.
struct TokenRefs {
  const int32_t* pos = nullptr;  // [batch] position of the first token
  const int32_t* cu = nullptr;
  int32_t n_tokens = 0, max_tokens = 1;
};

struct RopeLaunch {
  PageRefs pages;
  TokenRefs tok;
  const uint16_t *q = nullptr, *k = nullptr, *v = nullptr;
  uint16_t* q_out = nullptr;
  int64_t q_stride = 0, qo_stride = 0, k_stride = 0, v_stride = 0;
  const float* rope = nullptr;
  int32_t rope_positions = 0, rotary = 0, interleaved = 0;
  int32_t Hq = 0, Hkv = 0;
  uint16_t *k_pages = nullptr, *v_pages = nullptr;  // BF16 pages, or
  uint8_t* pages4 = nullptr;                        // 4-bit pages
  int32_t num_sms = 0;
  unsigned* err = nullptr;
};
cudaError_t launch_rope_append_bf16(const RopeLaunch& a, cudaStream_t stream);
cudaError_t launch_rope_append_int4(const RopeLaunch& a, cudaStream_t stream);
cudaError_t launch_rope_table(float* table, int32_t n_positions, int32_t rotary, double theta, cudaStream_t stream);

struct Read4Launch {
  PageRefs from, to;
  const int32_t *pos = nullptr, *count = nullptr;
  int32_t max_count = 0, Hkv = 0, num_sms = 0;
  const uint8_t* pages4 = nullptr;
  uint16_t *k_pages = nullptr, *v_pages = nullptr;
  unsigned* err = nullptr;
};
cudaError_t launch_int4_to_bf16(const Read4Launch& a, cudaStream_t stream);

// How the attention's work is laid out over blocks.
struct WindowPlan {
  int32_t items = 1;  // split kernel: blocks; tensor-core kernel: blocks that share one (tile pair, KV head)
  size_t off_records = 0, total = 0;  // workspace: counters, then the items' records; one size for all calls
};

struct WindowLaunch {
  PageRefs pages;
  TokenRefs tok;
  const uint16_t* q = nullptr;
  uint16_t* out = nullptr;
  int64_t q_stride = 0;
  const int32_t* ctx_len = nullptr;
  int32_t window = -1, sinks = 0;
  float sm_scale = 0.f;
  int32_t Hq = 0, Hkv = 0;
  const uint16_t *k_pages = nullptr, *v_pages = nullptr;  // BF16 pages, or
  const uint8_t* pages4 = nullptr;                        // 4-bit pages
  WindowPlan plan;
  uint8_t* workspace = nullptr;
  int32_t num_sms = 0;
  unsigned* err = nullptr;
};
constexpr int kCutBlocks = 2;  // blocks (split kernel) or items (tensor-core kernel) per SM that share out keys, at most
inline size_t window_counter_bytes(int num_sms) { return ((size_t)kCutBlocks * num_sms * sizeof(unsigned) + 255) & ~(size_t)255; }
WindowPlan plan_window(bool int4, int64_t rows, int Hq, int Hkv, int64_t max_keys, int num_sms);
cudaError_t launch_window_split(const WindowLaunch& a, cudaStream_t stream);

// Chunks and prompts over BF16 pages, on the tensor cores (records [items][256 rows][130])
// (the counters are the split kernel's; this one keeps off them)
WindowPlan plan_window_tc(int64_t batch, int64_t max_tokens, int Hq, int Hkv, int64_t max_keys, int num_sms);
cudaError_t launch_window_tc(const WindowLaunch& a, cudaStream_t stream);

}  // namespace oscar
