// C ABI of the gated delta rule: argument checks and launches.  Host code only.
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "errors.h"
#include "hyb_internal.h"
#include "k_delta.h"

using namespace hyb;

namespace {

// From this many tokens a sequence the chunks are faster than single steps: 4 sequences of 32 heads of 128 x 128, steps /
// chunks: 8 tokens 9.1 / 12.9 us, 12 12.1 / 13.0, 16 15.1 / 13.0, 64 51.7 / 13.5; 32 sequences: 8 tokens 62.3 / 91.4, 12 84.1 /
// 91.5, 16 106.5 / 91.8, 64 375 / 97; 4 heads, 4 sequences: 12 tokens 11.9 / 12.5, 16 14.9 / 12.5; heads of 64 x 64, 4 sequences:
// 12 8.8 / 10.3, 16 11.1 / 10.3.  Not so where heads of 64 x 64 are more than the SMs, whose steps share an SM and whose chunks
// do not: 32 sequences of 32, 16 tokens 25.4 / 66.4, 24 36.0 / 66.8.
constexpr int kChunksFrom = 14;

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool rows_ok(const void* p, int64_t stride, int64_t heads, int d) {
  return aligned(p, 16) && stride % 8 == 0 && stride >= heads * d && stride < ((int64_t)1 << 40);
}

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

}  // namespace

extern "C" int hyb_attn_delta_run(const hyb_attn_delta_state* st, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, const float* g, const float* beta,
                                  void* out, int64_t out_stride, const int32_t* cu_new, const int32_t* slots,
                                  int32_t batch, int32_t n_new, int32_t max_new, float scale, uint32_t* status,
                                  cudaStream_t stream) {
  const NvtxRange range(__func__);
  if (st == nullptr || !aligned(st->state, 16) || st->n_slots < 1 || st->n_k_heads < 1 || st->n_v_heads < 1) return HYB_EINVAL;
  if (st->n_v_heads % st->n_k_heads != 0) return HYB_EINVAL;
  if ((st->key_dim != 64 && st->key_dim != 128) || (st->value_dim != 64 && st->value_dim != 128)) return HYB_EINVAL;
  if (batch < 1 || n_new < 0 || n_new > (1 << 30) || max_new < 0 || max_new > n_new || (n_new > 0 && max_new < 1)) return HYB_EINVAL;
  if ((int64_t)batch * st->n_v_heads >= ((int64_t)1 << 31)) return HYB_EINVAL;
  if (slots == nullptr && batch > st->n_slots) return HYB_EINVAL;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return HYB_EINVAL;
  if (!aligned(cu_new, 4) || (slots != nullptr && !aligned(slots, 4)) || (status != nullptr && !aligned(status, 4))) return HYB_EINVAL;
  if (n_new == 0) return HYB_OK;
  if (!rows_ok(q, q_stride, st->n_k_heads, st->key_dim) || !rows_ok(k, k_stride, st->n_k_heads, st->key_dim) ||
      !rows_ok(v, v_stride, st->n_v_heads, st->value_dim) || !rows_ok(out, out_stride, st->n_v_heads, st->value_dim))
    return HYB_EINVAL;
  if (!aligned(g, 4) || !aligned(beta, 4)) return HYB_EINVAL;
  DeltaParams p{};
  p.state = st->state;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.g = g;
  p.beta = beta;
  p.out = static_cast<uint16_t*>(out);
  p.cu = cu_new;
  p.slots = slots;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = out_stride;
  p.B = batch;
  p.n_new = n_new;
  p.max_new = max_new;
  p.n_slots = st->n_slots;
  p.Hk = st->n_k_heads;
  p.Hv = st->n_v_heads;
  p.DK = st->key_dim;
  p.DV = st->value_dim;
  p.scale = scale > 0.f ? scale : 1.f / sqrtf((float)st->key_dim);
  p.status = status;
  const cudaError_t e = max_new < kChunksFrom ? launch_delta_steps(p, stream) : launch_delta_chunks(p, stream);
  return e == cudaSuccess ? HYB_OK : record_cuda_error(e);
}
