// The paged 8-bit cache: append with rotation, and attention over it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace hyb {

// Codes [n_pages][Hkv][P][D] and scales [n_pages][Hkv] of keys and values.
struct PagedCache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int32_t n_pages, Hkv, P;
};

// A step's sequences: new tokens [cu[b], cu[b + 1]) of sequence b, which has
// lens[b] tokens once they are counted.
struct PagedBatch {
  const int32_t* table;  // [B][mp] page of tokens [i * P, (i + 1) * P)
  const int32_t* cu;     // [B + 1]
  const int32_t* lens;   // [B]
  int32_t B, mp, n_new, max_new;
};

struct PagedAppendParams {
  PagedCache c;
  PagedBatch b;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;  // null: no query rotation
  uint16_t* q_out;
  const float* rope;  // [n_pos][rot] cosines then sines; null: no rotation
  int64_t k_stride, v_stride, q_stride, qo_stride;  // elements from token to token
  int32_t Hq, D, rot, n_pos;
  int32_t int8, half, interleaved;  // codes int8 (else e4m3); inputs fp16 (else bf16)
  int32_t pages_max;                // pages that one sequence's new tokens can touch
  int64_t kv_blocks;                // blocks of the cache part; the query part follows
  uint32_t* status;
};

struct PagedAttnParams {
  PagedCache c;
  PagedBatch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // [n_new][Hq] or null
  int64_t q_stride, out_stride;
  int32_t Hq, G, half, W, S;
  float scale;       // times log2(e)
  int32_t cluster;   // CTAs of a cluster that takes one unit (narrow form), or 0
  int32_t n_cta;     // CTAs that share the line of all units' stages
  int32_t quantum;   // stages that a CTA's part is a multiple of
  int32_t n_splits;  // parts of a row tile's stages: of each (wide form), of those from n_whole on (tcgen05)
  int32_t n_whole, row_tiles;  // tcgen05: row tiles taken whole; of each sequence and KV head
  float* ws;         // partial results
  uint32_t* status;
};

// Rows (new tokens x heads of a group) of one sequence and KV head that the
// narrow form takes in fp16, and those of a CTA of the wide form (fp16 only).
constexpr int kNarrowRows = 64;
constexpr int kWideRows = 64;
constexpr int kCtasPerSm = 3;
constexpr int kPagedMaxCluster = 8;
// Rows of a CTA of the form on tcgen05 (bf16 only).
constexpr int kMmaRows = 128;
constexpr int kMmaCtasPerSm = 2;

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s);
cudaError_t launch_paged_narrow(const PagedAttnParams& p, int D, int int8, int rows, cudaStream_t s);
cudaError_t launch_paged_mma(const PagedAttnParams& p, int D, int int8, cudaStream_t s);
cudaError_t launch_paged_wide(const PagedAttnParams& p, int D, int int8, cudaStream_t s);

// Joins of the parts that several CTAs left: of the line of 128-token tiles with `rows` rows a unit; of n_splits
// parts of every row; of row tiles from n_whole on.
cudaError_t launch_paged_join(const PagedAttnParams& p, int D, int rows, cudaStream_t s);
cudaError_t launch_paged_join_tiles(const PagedAttnParams& p, int D, cudaStream_t s);

}  // namespace hyb
