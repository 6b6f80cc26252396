// k_kv4.cuh -- arguments and launchers of the decode step's attention block (kv4_attn.h):
// step tables, query/key norm with rotation, the MXFP4 cache's rows, attention over it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kv4 {

constexpr int kMaxReqs = 1024;
constexpr int kMaxPage = 1024;
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxKvHeads = 256;

// Bits of a *status word (MOE_KV4_STATUS_* in kv4_attn.h).
enum : int32_t {
  kStatusTimeout = 4,
  kStatusBadLength = 16,
  kStatusNoPages = 32,
  kStatusRows = 64,
  kStatusBadSlot = 128,
  kStatusBadPage = 256,
};

struct TablesArgs {
  int reqs, max_rows, page, n_free, width;
  uint64_t page_magic;  // ceil(2^64 / page): a length / page by a multiply
  int64_t stride;
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* row_starts;
  int32_t* kv_lens;
  int32_t* positions;
  int64_t* slots;
  int32_t* used;
  int32_t* status;
};
cudaError_t launch_step_tables(const TablesArgs& a, cudaStream_t st);

struct RopeArgs {
  int rows, hq, hk, D, rot, interleaved;
  float eps;
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  int64_t ldq, ldk, ldqo, ldko;
  const uint16_t* gq;
  const uint16_t* gk;
  const int32_t* pos;
  const float* freq;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st);

struct RowsArgs {
  int rows, heads, D, page;
  int64_t n_slots;      // n_pages * page
  uint64_t page_magic;  // ceil(2^64 / page): slot / page by a multiply
  int units;            // of a row's heads (set by the launch)
  uint64_t unit_magic;  // ceil(2^64 / units) (of two units and more)
  uint8_t* cache;
  uint16_t* k;  // read by the append, written by the read
  uint16_t* v;
  int64_t ldk, ldv;
  const int64_t* slots;
  int32_t* status;
};
cudaError_t launch_kv4_append(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_kv4_read(const RowsArgs& a, cudaStream_t st);

struct AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  const uint8_t* cache;
  int64_t n_pages;
  int rows, reqs, heads, G, D;  // heads: kv heads; G: query heads of each
  int page_tiles;               // page_size / 16
  uint64_t page_magic;          // ceil(2^34 / page_tiles): tile / page_tiles by a multiply
  const int32_t* table;
  int64_t stride;
  int max_len;  // the tokens that a table row can hold
  const int32_t* row_starts;
  const int32_t* kv_lens;
  float scale_log2;  // softmax scale * log2(e)
  int window, sinks;
  uint16_t* out;
  int64_t ldo;
  float* part;  // workspace: [2 ctas][RN][D] averages, then [2 ctas][RN][2] (max, sum)
  int ctas;
  int stall;  // failure tests: a barrier of CTA 0 that expects one arrival more than is sent (negative: none)
  int32_t* status;
};
// Query rows of one work item for calls with up to `max_new` rows of a request.
int attn_rows_per_item(int G, int max_new);
// CTAs of the attention launch on the current device (0 on a CUDA error, left in *err).
int attn_ctas(cudaError_t* err);
size_t attn_workspace_bytes(int D, int rn, int ctas);
cudaError_t launch_kv4_attention(const AttnArgs& a, int rn, cudaStream_t st);

}  // namespace kv4
