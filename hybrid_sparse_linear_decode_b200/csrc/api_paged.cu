// C ABI of the paged 8-bit cache: argument checks, work splits, launches.  Host code only.
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>

#include "errors.h"
#include "hyb_internal.h"
#include "k_paged.h"

using namespace hyb;

namespace {

// The splits are planned for this many SMs; a device with fewer still runs them.
constexpr int kSms = 148;

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Shapes only (what the workspace size depends on).
bool shapes_ok(const hyb_attn_paged_cache* c, const hyb_attn_paged_batch* b) {
  if (c == nullptr || b == nullptr) return false;
  if (c->n_pages < 1 || c->n_kv_heads < 1) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->page_size < 16 || c->page_size > 256 || c->page_size % 16 != 0) return false;
  if (c->code != HYB_CODE_E4M3 && c->code != HYB_CODE_INT8) return false;
  // the tcgen05 form counts the rows of keys in 32 bits (64 bytes each at least: 256 GB)
  if ((int64_t)c->n_pages * c->n_kv_heads >= 0xffffffffll / c->page_size) return false;
  if (b->batch < 1 || b->table_stride < 1 || (int64_t)b->table_stride * c->page_size > ((int64_t)1 << 30)) return false;
  if ((int64_t)b->batch * c->n_kv_heads > 65535) return false;
  // 32-token stages of all sequences and KV heads are counted in 31 bits
  if ((int64_t)b->batch * c->n_kv_heads * ((int64_t)b->table_stride * c->page_size / 32 + 2) >= ((int64_t)1 << 31)) return false;
  if (b->n_new < 0 || b->n_new > (1 << 30) || b->max_new < 0 || b->max_new > b->n_new || b->max_len < 0) return false;
  return b->n_new == 0 || b->max_new > 0;
}

bool pointers_ok(const hyb_attn_paged_cache* c, const hyb_attn_paged_batch* b) {
  return aligned(c->k_codes, 16) && aligned(c->v_codes, 16) && aligned(c->k_scales, 4) && aligned(c->v_scales, 4) &&
         aligned(b->page_table, 4) && aligned(b->cu_new, 4) && aligned(b->kv_lens, 4) &&
         (b->status == nullptr || aligned(b->status, 4));
}

PagedCache cache_of(const hyb_attn_paged_cache* c) {
  return PagedCache{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scales, c->v_scales,
                    c->n_pages, c->n_kv_heads, c->page_size};
}
PagedBatch batch_of(const hyb_attn_paged_batch* b) {
  return PagedBatch{b->page_table, b->cu_new, b->kv_lens, b->batch, b->table_stride, b->n_new, b->max_new};
}

// Rows of `heads` heads of head_dim elements, `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int64_t heads, int d, int64_t unit) {
  return aligned(p, unit * 2) && stride % unit == 0 && stride >= heads * d && stride < ((int64_t)1 << 40);
}

struct Plan {
  enum Form { kNarrow, kWide, kMma } form;
  int rows;      // of the line's units: narrow 8, 16, 32 or 64, mma 128; 0 with splits
  int cluster;   // CTAs a unit (narrow), or 0
  int n_cta;     // line
  int n_splits;  // otherwise
  int64_t n_whole, row_tiles;  // mma: row tiles taken whole; of a unit
  size_t bytes;
};

// Up to kNarrowMost rows a KV head: narrow, 8 or 16 rows a warp, bound by the codes' bytes.  More: bf16 on tcgen05, in
// whose 128 rows one conversion of the codes serves all; fp16, whose weights go in as two parts, on the warps' own
// products (narrow up to 64 rows, then wide).  8 sequences of up to 32K tokens, 8 KV heads of 128, 4 rows a token, narrow /
// tcgen05: 20 rows 151 / 161 us, 32 rows 158 / 163; heads of 64, int8: 102 / 136, 105 / 138; 2 KV heads: 52 / 53, 57 / 53;
// one sequence of 4096: 14.9 / 14.1, 15.8 / 16.1.  48 rows took 294 / 208 and 64 rows 303 / 204 when measured; tcgen05 takes
// 199 and 194 now.
// While a sequence's rows fit one tile the CTAs share the line of all tiles; more rows, and few row tiles, cut each row
// tile's tokens into as many parts as the SMs hold at once, each of at least kLeastTokens (128 tokens of one sequence,
// parts of at least 128 / 256 / 512 / 1024 tokens: of 1024 tokens 26 / 23 / 28 / 34 us, of 2048 41 / 30 / 29 / 40).
constexpr int kNarrowMost = 32;
constexpr int kLeastTokens = 256;
// On tcgen05, row tiles that fill the SMs more than half, or come behind full turns of them, go in parts of at least
// kLeastTail tokens (512 / 1024 / 2048 / whole, when a tile took 5 % more than it does: 2047 tokens of 10001 608 / 608 / 608 /
// 639 us, 1300 of 8192 335 / 334 / 325 / 440, 1300 of 4096 171 / 172 / 189 / 211, 700 of 4096 141 / 129 / 144 / 144, 2048 of
// 2048 136 / 98 / 98 / 98).
constexpr int kLeastTail = 1024;
// The narrow form by clusters or by the line: a cluster's CTA takes stages / CTAs stages of 32 tokens; on the line it
// takes an equal share of all, and the second launch that joins the parts costs about kLineStages stages' time.  (What a
// length gives to clusters, every shorter one does too, so a window needs no workspace that no window does not.)  One
// token each, 4096 tokens, 8 KV heads of 128, clusters / line: 8 sequences 18.6 / 21.4 us, 16 28.8 / 31.8; 32 sequences of
// 2048 34.9 / 32.4, of 1024 20.4 / 22.0; 64 of 1024 35.1 / 36.1; 8 of 16384 49.2 / 52.2, of 32768 94.1 / 93.4.  Heads of 64,
// int8, fp16: 8 of 4096 15.1 / 17.0, 32 of 2048 28.5 / 27.4, 64 of 1024 27.2 / 30.8; 2 KV heads of 8 query heads each: 16 of
// 4096 16.4 / 16.3, 32 of 2048 13.3 / 16.5; one KV head: 64 of 1024 9.7 / 12.1.  Clusters above 8 are not used: 4 sequences
// of 4096 in clusters of 13 20.2 / 15.5, 2 in clusters of 16 11.6 / 11.9, 1 of 16384 17.7 / 16.4.
constexpr int64_t kLineStages = 8;

Plan make_plan(const hyb_attn_paged_cache* c, const hyb_attn_paged_batch* b, int Hq, int window, int sink, int type) {
  Plan p{};
  const int G = Hq / c->n_kv_heads;
  const int64_t units = (int64_t)b->batch * c->n_kv_heads;
  const int64_t rows = (int64_t)b->max_new * G;
  int64_t len = std::min<int64_t>(b->max_len, (int64_t)b->table_stride * c->page_size);
  if (window > 0) len = std::min<int64_t>(len, (int64_t)window + sink + b->max_new + 64);
  const size_t row_bytes = (size_t)(c->head_dim + 4) * sizeof(float);
  const bool mma = rows > kNarrowMost && type == HYB_TYPE_BF16;
  p.form = mma ? Plan::kMma : rows <= kNarrowRows ? Plan::kNarrow : Plan::kWide;
  const int tile = mma ? kMmaRows : kWideRows;
  if (p.form == Plan::kNarrow || (mma && rows <= tile)) {
    const int64_t stage = mma ? 128 : 32, warps = mma ? 1 : 4;
    const int64_t stages = std::max<int64_t>(1, (len + stage - 1) / stage);
    p.rows = mma ? tile : rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    if (!mma) {
      // each CTA's part of a unit: a stage for each of its warps at least, all units' CTAs on the SMs at once if they can
      const int64_t slots = kSms * kCtasPerSm, n = std::min<int64_t>(std::max<int64_t>(1, slots / units), (stages + 3) / 4);
      if (n <= kPagedMaxCluster && stages * (slots - std::min(slots, units * n)) <= kLineStages * n * slots) {
        p.cluster = (int)n;
        return p;
      }
    }
    p.n_cta = (int)std::max<int64_t>(1, std::min<int64_t>(kSms * (mma ? kMmaCtasPerSm : kCtasPerSm), (units * stages + warps - 1) / warps));
    p.bytes = (size_t)2 * p.n_cta * p.rows * row_bytes;
  } else {
    p.row_tiles = (rows + tile - 1) / tile;
    const int64_t tiles = units * p.row_tiles, all = kSms * (mma ? kMmaCtasPerSm : kCtasPerSm);
    int64_t n = std::max<int64_t>(1, std::min<int64_t>({all / tiles, len / kLeastTokens, 64}));
    if (!mma) {
      if (b->max_new > 65535 || b->batch > 65535) n = 1;  // the join's grid
      p.n_splits = (int)n;
      p.bytes = n > 1 ? (size_t)n * b->n_new * Hq * row_bytes : 0;
    } else {
      // tiles behind the last full turn of the SMs: the parts that take the fewest turns of a part's length
      const int64_t rest = tiles % all;
      if (2 * rest > all)
        for (int64_t i = 2; i <= std::min<int64_t>(8, len / kLeastTail); ++i)
          if (((rest * i + all - 1) / all) * n < ((rest * n + all - 1) / all) * i) n = i;
      if (2 * rest <= all && tiles > all && rest > 0)
        n = std::max<int64_t>(1, std::min<int64_t>({all / rest, len / kLeastTail, 8}));
      p.n_splits = (int)n;
      p.n_whole = n > 1 ? tiles - rest : tiles;
      p.bytes = n > 1 ? (size_t)(rest * n) * tile * row_bytes : 0;
    }
  }
  return p;
}

}  // namespace

extern "C" {

int hyb_attn_paged_append(const hyb_attn_paged_cache* cache, const hyb_attn_paged_batch* batch, int32_t type,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* rope,
                          int32_t n_pos, int32_t rot_dim, int32_t interleaved, const void* q, int64_t q_stride,
                          void* q_out, int64_t q_out_stride, int32_t n_q_heads, cudaStream_t stream) {
  const NvtxRange range(__func__);
  if (!shapes_ok(cache, batch) || !pointers_ok(cache, batch)) return HYB_EINVAL;
  if (type != HYB_TYPE_BF16 && type != HYB_TYPE_FP16) return HYB_EINVAL;
  const int d = cache->head_dim;
  if ((q == nullptr) != (q_out == nullptr)) return HYB_EINVAL;
  if (rope != nullptr && (!aligned(rope, 16) || n_pos < 1 || rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0))
    return HYB_EINVAL;
  if (batch->n_new == 0) return HYB_OK;
  if (!rows_ok(k, k_stride, cache->n_kv_heads, d, 8) || !rows_ok(v, v_stride, cache->n_kv_heads, d, 8)) return HYB_EINVAL;
  if (q != nullptr) {
    if (n_q_heads < 1 || !rows_ok(q, q_stride, n_q_heads, d, 8) || !rows_ok(q_out, q_out_stride, n_q_heads, d, 8))
      return HYB_EINVAL;
    if (q == q_out && q_stride != q_out_stride) return HYB_EINVAL;
  }
  PagedAppendParams p{};
  p.c = cache_of(cache);
  p.b = batch_of(batch);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q = static_cast<const uint16_t*>(q);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.rope = rope;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.qo_stride = q_out_stride;
  p.Hq = q != nullptr ? n_q_heads : 0;
  p.D = d;
  p.rot = rope != nullptr ? rot_dim : 0;
  p.n_pos = n_pos;
  p.int8 = cache->code == HYB_CODE_INT8;
  p.half = type == HYB_TYPE_FP16;
  p.interleaved = interleaved != 0;
  p.pages_max = (batch->max_new - 1 + cache->page_size - 1) / cache->page_size + 1;
  p.kv_blocks = (int64_t)batch->batch * p.pages_max * cache->n_kv_heads * 2;
  p.status = batch->status;
  if (p.kv_blocks + (int64_t)batch->n_new * (p.Hq + 3) / 4 * 8 / 32 + 1 >= ((int64_t)1 << 31)) return HYB_EINVAL;
  const cudaError_t e = launch_paged_append(p, stream);
  return e == cudaSuccess ? HYB_OK : record_cuda_error(e);
}

size_t hyb_attn_paged_workspace_size(const hyb_attn_paged_cache* cache, const hyb_attn_paged_batch* batch,
                                     int32_t n_q_heads) {
  if (!shapes_ok(cache, batch) || n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0 || batch->n_new == 0) return 0;
  return std::max(make_plan(cache, batch, n_q_heads, 0, 0, HYB_TYPE_BF16).bytes, make_plan(cache, batch, n_q_heads, 0, 0, HYB_TYPE_FP16).bytes);
}

int hyb_attn_paged_attend(const hyb_attn_paged_cache* cache, const hyb_attn_paged_batch* batch, int32_t type,
                          const void* q, int64_t q_stride, void* out, int64_t out_stride, float* lse,
                          int32_t n_q_heads, int32_t window, int32_t n_sink, float scale, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  const NvtxRange range(__func__);
  if (!shapes_ok(cache, batch) || !pointers_ok(cache, batch)) return HYB_EINVAL;
  if (type != HYB_TYPE_BF16 && type != HYB_TYPE_FP16) return HYB_EINVAL;
  if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0) return HYB_EINVAL;
  if (window < 0 || n_sink < 0 || !(scale >= 0.f) || !std::isfinite(scale)) return HYB_EINVAL;
  const int d = cache->head_dim;
  if (batch->n_new == 0) return HYB_OK;
  if (!rows_ok(q, q_stride, n_q_heads, d, 8) || !rows_ok(out, out_stride, n_q_heads, d, 4)) return HYB_EINVAL;
  if (lse != nullptr && !aligned(lse, 4)) return HYB_EINVAL;
  if ((int64_t)batch->max_new * (n_q_heads / cache->n_kv_heads) > ((int64_t)1 << 30)) return HYB_EINVAL;
  const Plan plan = make_plan(cache, batch, n_q_heads, window, n_sink, type);
  if (plan.form == Plan::kMma && (plan.row_tiles * batch->batch * cache->n_kv_heads) * plan.n_splits >= ((int64_t)1 << 31)) return HYB_EINVAL;
  if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes)) return HYB_ESCRATCH;
  if (plan.bytes > 0 && !aligned(workspace, 16)) return HYB_EINVAL;
  PagedAttnParams p{};
  p.c = cache_of(cache);
  p.b = batch_of(batch);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.Hq = n_q_heads;
  p.G = n_q_heads / cache->n_kv_heads;
  p.half = type == HYB_TYPE_FP16;
  p.W = window;
  p.S = window > 0 ? n_sink : 0;
  p.scale = (scale > 0.f ? scale : 1.f / sqrtf((float)d)) * 1.44269504088896341f;
  p.cluster = plan.cluster;
  p.n_cta = plan.n_cta;
  p.quantum = plan.form == Plan::kMma ? 1 : 4;
  p.n_splits = plan.n_splits;
  p.n_whole = (int)plan.n_whole;
  p.row_tiles = (int)plan.row_tiles;
  p.ws = static_cast<float*>(workspace);
  p.status = batch->status;
  const int int8 = cache->code == HYB_CODE_INT8;
  const cudaError_t e = plan.form == Plan::kMma      ? launch_paged_mma(p, d, int8, stream)
                        : plan.form == Plan::kNarrow ? launch_paged_narrow(p, d, int8, plan.rows, stream)
                                                     : launch_paged_wide(p, d, int8, stream);
  return e == cudaSuccess ? HYB_OK : record_cuda_error(e);
}

}  // extern "C"
