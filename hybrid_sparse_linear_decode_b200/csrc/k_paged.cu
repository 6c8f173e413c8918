// Attention over the paged 8-bit cache, and the append that fills it.
#include <cuda_fp16.h>

#include <cfloat>

#include "hyb_device.cuh"
#include "k_paged.h"

namespace hyb {
namespace {

__device__ __forceinline__ void raise(uint32_t* status, uint32_t bit) {
  if (status != nullptr) atomicOr(status, bit);
}

// ---- 16-bit inputs ----------------------------------------------------------------------------
__device__ __forceinline__ float in_lo(uint32_t w, bool half) {
  return half ? __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))) : bf16_lo(w);
}
__device__ __forceinline__ float in_hi(uint32_t w, bool half) {
  return half ? __half2float(__ushort_as_half((unsigned short)(w >> 16))) : bf16_hi(w);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, bool half) {
  return half ? pack_half(lo, hi) : pack_bf16(lo, hi);
}

// ---- a sequence of the step --------------------------------------------------------------------
struct Seq {
  int t0, n, len;  // first row, new tokens, tokens in all
};

// Reads a sequence's ranges and holds them within what the caller said: rows
// within [0, n_new), at most max_new of them, a length within the page table.
__device__ __forceinline__ Seq read_seq(const PagedBatch& b, int i, int P, bool* bad) {
  Seq s;
  const int c0 = b.cu[i], c1 = b.cu[i + 1], len = b.lens[i];
  s.t0 = min(max(c0, 0), b.n_new);
  const int t1 = min(max(c1, s.t0), b.n_new);
  s.n = min(t1 - s.t0, b.max_new);
  const int64_t cap = (int64_t)b.mp * P;
  s.len = (int)min((int64_t)max(len, 0), cap);
  *bad = s.t0 != c0 || s.n != c1 - c0 || s.len != len;
  return s;
}

// ================================================================================================
// Append
// ================================================================================================
//
// One CTA takes the new tokens that fall into one page of one sequence, for one
// KV head and for keys or values: it holds them rotated in registers (4 rows of
// 16 channels a thread), reduces their largest magnitude, settles the page's
// scale, rewrites the codes that the page already holds if the scale grew, and
// writes the new codes.  So each input is read once and each code written once.

constexpr int kAppendRows = 4;  // rows a thread holds

// a * c - b * s, correctly rounded for 16-bit a and b but for ties within 2^-45:
// the products' rounding errors are exact (fma), their difference's too (two-sum).
__device__ __forceinline__ float diff_of_products(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float q = __fmul_rn(b, s), qe = __fmaf_rn(b, s, -q);
  const float d = __fsub_rn(p, q);
  const float bb = __fsub_rn(d, p);
  const float de = __fsub_rn(__fsub_rn(p, __fsub_rn(d, bb)), __fadd_rn(q, bb));
  const float r = __fadd_rn(d, __fadd_rn(de, __fsub_rn(pe, qe)));
  // an infinite or NaN input leaves NaN in the error terms: take the plain value there
  return r == r ? r : d;
}

__device__ __forceinline__ float scale_for(float amax, bool int8) {
  if (int8) return fmaxf(__fdiv_rn(amax, 127.f), 1.17549435e-38f);
  // the smallest power of two x in [2^-126, 2^126] with amax <= 448 x:
  // 448 = 1.75 * 2^8, so x = 2^(e - 8) or the next for amax = m 2^e, 1 <= m < 2
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, -126), 126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Code of y (already divided by the scale): nearest, ties to even, saturating;
// NaN becomes 0.
__device__ __forceinline__ uint32_t code2(float lo, float hi, bool int8) {
  lo = lo == lo ? lo : 0.f;
  hi = hi == hi ? hi : 0.f;
  if (int8) {
    const int a = __float2int_rn(fminf(fmaxf(lo, -127.f), 127.f));
    const int b = __float2int_rn(fminf(fmaxf(hi, -127.f), 127.f));
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
  }
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t code4(const float* y, float inv, bool int8) {
  return code2(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv), int8) |
         (code2(__fmul_rn(y[2], inv), __fmul_rn(y[3], inv), int8) << 16);
}
// The value a code stands for, without its scale (e4m3's NaN codes stay NaN).
__device__ __forceinline__ float value_of(uint32_t byte, bool int8) {
  if (int8) return (float)(int)(int8_t)byte;
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// The 16 channels of a lane: two runs of 8 that hold whole pairs.  Of the first
// rot channels, half-split pairs (i, i + rot / 2) take a run from each half;
// interleaved pairs and the channels past rot take 16 in a row.
struct Runs {
  int c0, c1, angle;  // first channels of the runs; first pair, or -1 outside the rotation
};
__device__ __forceinline__ Runs lane_runs(int j, int rot, bool interleaved) {
  Runs r;
  const bool turned = j < rot / 16;
  r.angle = turned ? 8 * j : -1;
  r.c0 = turned && !interleaved ? 8 * j : 16 * j;
  r.c1 = turned && !interleaved ? rot / 2 + 8 * j : 16 * j + 8;
  return r;
}
__device__ __forceinline__ void load_runs(const uint16_t* row, const Runs& r, bool half, float* x) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + r.c0));
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(row + r.c1));
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = in_lo(w[i], half);
    x[2 * i + 1] = in_hi(w[i], half);
  }
}
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int rot, int at) {
  const float4* c = reinterpret_cast<const float4*>(row + at);
  const float4* s = reinterpret_cast<const float4*>(row + rot / 2 + at);
  const float4 x = __ldg(c), y = __ldg(c + 1), z = __ldg(s), w = __ldg(s + 1);
  a.c[0] = x.x, a.c[1] = x.y, a.c[2] = x.z, a.c[3] = x.w, a.c[4] = y.x, a.c[5] = y.y, a.c[6] = y.z, a.c[7] = y.w;
  a.s[0] = z.x, a.s[1] = z.y, a.s[2] = z.z, a.s[3] = z.w, a.s[4] = w.x, a.s[5] = w.y, a.s[6] = w.z, a.s[7] = w.w;
}
template <bool EXACT>
__device__ __forceinline__ void turn(float* x, const Angles& a, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& u = interleaved ? x[2 * i] : x[i];
    float& w = interleaved ? x[2 * i + 1] : x[8 + i];
    const float p = u, q = w;
    if (EXACT) {
      u = diff_of_products(p, a.c[i], q, a.s[i]);
      w = diff_of_products(q, a.c[i], -p, a.s[i]);
    } else {  // an output of 16 bits: one rounding of a product's error is enough
      const float m = __fmul_rn(q, a.s[i]), n = __fmul_rn(p, a.s[i]);
      u = __fsub_rn(__fmaf_rn(p, a.c[i], -m), __fmaf_rn(q, a.s[i], -m));
      w = __fadd_rn(__fmaf_rn(q, a.c[i], n), __fmaf_rn(p, a.s[i], -n));
    }
  }
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(512) paged_append_kernel(const PagedAppendParams p) {
  const bool half = p.half != 0, int8 = p.int8 != 0;
  const int lanes = p.D / 16;  // lanes of a row: 4 or 8
  const int P = p.c.P;

  if ((int64_t)blockIdx.x >= p.kv_blocks) {
    // The query part: a thread turns the same channels of 4 heads of one token.
    const int groups = (p.Hq + 3) / 4;
    const int64_t at = ((int64_t)blockIdx.x - p.kv_blocks) * blockDim.x + threadIdx.x;
    const int j = (int)(at % lanes);
    const int64_t rest = at / lanes;
    const int hg = (int)(rest % groups);
    const int64_t t = rest / groups;
    if (t >= p.b.n_new) return;
    // the token's sequence: the last b with cu[b] <= t
    int lo = 0, hi = p.b.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.b.cu[mid] <= t) lo = mid; else hi = mid;
    }
    bool bad;
    const Seq s = read_seq(p.b, lo, P, &bad);
    if (t < s.t0 || t >= s.t0 + s.n) return;  // a row behind the last sequence
    const Runs r = lane_runs(j, p.rot, INTERLEAVED);
    Angles a;
    if (r.angle >= 0) {
      const int pos = s.len - s.n + (int)(t - s.t0);
      if (pos < 0 || pos >= p.n_pos) raise(p.status, HYB_STATUS_BAD_LENGTH);
      load_angles(a, p.rope + (int64_t)min(max(pos, 0), p.n_pos - 1) * p.rot, p.rot, r.angle);
    }
    const int heads = min(4, p.Hq - hg * 4);
    float x[4][16];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (h < heads) load_runs(p.q + t * p.q_stride + (int64_t)(hg * 4 + h) * p.D, r, half, x[h]);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (h >= heads) break;
      if (r.angle >= 0) turn<false>(x[h], a, INTERLEAVED);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_out(x[h][2 * i], x[h][2 * i + 1], half);
      uint16_t* row = p.q_out + t * p.qo_stride + (int64_t)(hg * 4 + h) * p.D;
      *reinterpret_cast<uint4*>(row + r.c0) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(row + r.c1) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return;
  }

  // The cache part: blocks ordered by sequence, page, KV head, keys / values.
  uint32_t bi = blockIdx.x;
  const bool values = bi & 1;
  bi >>= 1;
  const int h = (int)(bi % (uint32_t)p.c.Hkv);
  bi /= (uint32_t)p.c.Hkv;
  const int pi = (int)(bi % (uint32_t)p.pages_max);
  const int b = (int)(bi / (uint32_t)p.pages_max);
  bool bad;
  const Seq s = read_seq(p.b, b, P, &bad);
  if (bad && pi == 0 && h == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
  const int start = s.len - s.n;  // position of the first new token
  const int first = max(start, 0);
  if (start < 0 && pi == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
  const int pg = first / P + pi;  // page of the sequence
  const int lo = max(pg * P, first), hi = (int)min((int64_t)(pg + 1) * P, (int64_t)s.len);
  if (lo >= hi) return;
  const int page = p.b.table[(int64_t)b * p.b.mp + pg];
  if (page < 0 || page >= p.c.n_pages) {
    if (threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_PAGE);
    return;
  }
  float* scale_at = (values ? p.c.vs : p.c.ks) + (int64_t)page * p.c.Hkv + h;
  uint8_t* codes = (values ? p.c.v : p.c.k) + ((int64_t)page * p.c.Hkv + h) * P * p.D;
  const int older = lo - pg * P;  // tokens that the page held before
  const float was = older > 0 ? *scale_at : 0.f;

  const int j = threadIdx.x % lanes, row0 = threadIdx.x / lanes, step = blockDim.x / lanes;
  const Runs r = lane_runs(j, values ? 0 : p.rot, INTERLEAVED);
  const uint16_t* in = values ? p.v : p.k;
  const int64_t stride = values ? p.v_stride : p.k_stride;
  float x[kAppendRows][16];
  float amax = 0.f;
  bool odd = false;  // an infinite or NaN value among them
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos < hi) load_runs(in + (int64_t)(s.t0 + pos - start) * stride + (int64_t)h * p.D, r, half, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos >= hi) continue;
    if (r.angle >= 0) {
      Angles a;
      if (pos >= p.n_pos) raise(p.status, HYB_STATUS_BAD_LENGTH);
      load_angles(a, p.rope + (int64_t)min(pos, p.n_pos - 1) * p.rot, p.rot, r.angle);
      turn<true>(x[i], a, INTERLEAVED);
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float y = fabsf(x[i][c]);
      const bool fine = y <= FLT_MAX;
      amax = fmaxf(amax, fine ? y : 0.f);
      odd |= !fine;
    }
  }
  if (odd) raise(p.status, HYB_STATUS_NONFINITE);
  __shared__ float part[16];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, part[w]);
  const float need = scale_for(amax, int8);
  // a scale only grows while the page holds tokens (a NaN left there is replaced)
  const float now = older > 0 && was >= need ? was : need;
  const float inv = __fdiv_rn(1.f, now);
  if (older > 0 && now != was) {
    const float ratio = __fmul_rn(was, inv);
    const int words = older * p.D / 4;
    for (int w = threadIdx.x; w < words; w += blockDim.x) {
      uint32_t* at = reinterpret_cast<uint32_t*>(codes) + w;
      const uint32_t c = *at;
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = value_of((c >> (8 * i)) & 0xffu, int8);
      *at = code4(y, ratio, int8);
    }
  }
  if (threadIdx.x == 0 && !(older > 0 && now == was)) *scale_at = now;
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos >= hi) continue;
    uint8_t* row = codes + (int64_t)(pos - pg * P) * p.D;
    *reinterpret_cast<uint2*>(row + r.c0) = make_uint2(code4(x[i], inv, int8), code4(x[i] + 4, inv, int8));
    *reinterpret_cast<uint2*>(row + r.c1) = make_uint2(code4(x[i] + 8, inv, int8), code4(x[i] + 12, inv, int8));
  }
}

// ================================================================================================
// Attention
// ================================================================================================
//
// With codes c and scales: k_t = ks c_t, v_t = vs c_t (ks, vs of t's page).  A
// row's logits in powers of two are z_t = (q . c_t) ks scale log2(e), its output
// sum_t 2^(z_t - m) vs c_t / sum_t 2^(z_t - m) with the running maximum m.
//
// Codes become f16 exactly.  Query rows are divided by a power of two that puts
// their largest element in [1, 2), so bf16 queries become f16 with no loss above
// 2^-17 of that element.  Weights are stored as f16(2^(z - m + 15) vs / ref) with
// ref a power of two that is at least every scale so far: at most 2^15, and full
// 11 bits down to 2^-29 of the largest, which is one rounding of 2^-12 a weight,
// below the output type's own.  All sums are in 32 bits.
//
// Matrix form (mma.m16n8k16): S = Q C_k^T with 16 rows of queries and 8 tokens,
// O = P C_v.  The channel and token orders inside a k-step are free as long as
// both operands agree, so a lane reads its 16 bytes of a token's codes at once
// and each 4-byte word of them is one k-step's fragment after two conversions.

constexpr int kStageTokens = 32;
constexpr int kWarps = 4;

template <int D>
struct StageGeo {
  static constexpr int kBytes = kStageTokens * D * 2 + 32;  // K codes, V codes, scales and flags
};
// Narrow form: CTAs an SM (registers: 168 or 255 a thread) and stages of each warp's ring.
template <int D, int MT>
struct NarrowGeo {
  static constexpr int kCtas = narrow_ctas_per_sm(MT);
  static constexpr int kStages = D == 128 ? (MT == 1 ? 2 : 3) : (MT == 1 ? 4 : 5);
};

// 16-byte column of a stage row, moved so that the reads of both products meet
// no bank twice: a quarter-warp reads 4 columns of two neighbouring rows (K) or 2
// columns of rows 2 apart (V).
template <int D>
__device__ __forceinline__ int swz(int row, int col) {
  if (D == 128) return col ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2));
  return col ^ (((row >> 1) & 1) << 1);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four codes to two f16 pairs (bytes 0, 1 and bytes 2, 3), exactly.
template <bool INT8>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (INT8) {
    // 1024 + (c + 128) has the byte c + 128 as its low bits; c + 128 is c with the sign bit flipped
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  } else {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Exponent field of the power of two at or above x (0 <= x <= 2^126, the scales'
// range), at least 2^-126; infinity and NaN give 2^126, and the weights take them on.
__device__ __forceinline__ uint32_t pow2_above(float x) {
  const uint32_t u = __float_as_uint(x);
  return min(max((u >> 23) + ((u & 0x7fffffu) ? 1u : 0u), 1u), 253u);
}
__device__ __forceinline__ float pow2_of(uint32_t e) { return __uint_as_float(e << 23); }

// Where the visible tokens of a row tile lie: sinks [0, sink), then [lo, hi)
// from a multiple of 16; 32-token stages, the sinks' first.
struct Span {
  int sink, lo, hi, sink_stages, stages;
};
__device__ __forceinline__ Span make_span(int pos_min, int pos_max, int W, int S) {
  Span s;
  s.hi = pos_max + 1;
  s.lo = W > 0 ? max(pos_min - W + 1, 0) & ~15 : 0;
  s.sink = W > 0 ? min(S, s.lo) : 0;
  s.sink_stages = (s.sink + kStageTokens - 1) / kStageTokens;
  s.stages = s.sink_stages + (max(s.hi - s.lo, 0) + kStageTokens - 1) / kStageTokens;
  return s;
}
__device__ __forceinline__ void stage_range(const Span& s, int st, int& base, int& end) {
  if (st < s.sink_stages) {
    base = st * kStageTokens;
    end = min(base + kStageTokens, s.sink);
  } else {
    base = s.lo + (st - s.sink_stages) * kStageTokens;
    end = min(base + kStageTokens, s.hi);
  }
}

// Pages of a stage's two 16-token groups (-1: none, or out of range).
struct StagePages {
  int p0, p1, o0, o1;  // pages, and the groups' first tokens within them
};
__device__ __forceinline__ StagePages stage_pages(const PagedAttnParams& p, const int32_t* table, int base, int end,
                                                  uint32_t magic) {
  // base is a multiple of 16, and so is P: base / P = (base / 16) / (P / 16) by a multiplication
  // (magic = ceil(2^32 / (P / 16)) is exact below 2^28 for a divisor of at most 16)
  StagePages g;
  const int P = p.c.P;
  const uint32_t a = (uint32_t)base >> 4, b = a + 1;
  const int ia = P == 16 ? (int)a : (int)__umulhi(a, magic), ib = P == 16 ? (int)b : (int)__umulhi(b, magic);
  g.p0 = base < end ? __ldg(table + ia) : -1;
  g.p1 = base + 16 < end ? __ldg(table + ib) : -1;
  g.o0 = base - ia * P;
  g.o1 = base + 16 - ib * P;
  if ((base < end && (uint32_t)g.p0 >= (uint32_t)p.c.n_pages) ||
      (base + 16 < end && (uint32_t)g.p1 >= (uint32_t)p.c.n_pages)) {
    raise(p.status, HYB_STATUS_BAD_PAGE);
    if ((uint32_t)g.p0 >= (uint32_t)p.c.n_pages) g.p0 = -1;
    if ((uint32_t)g.p1 >= (uint32_t)p.c.n_pages) g.p1 = -1;
  }
  return g;
}

// Starts the copies of a stage: N threads (this one is number `me`) take its
// 16-byte pieces in turn.  Tokens at or past `end` and of missing pages are
// filled with zeros, so nothing behind a sequence's end is read.
template <int D, int N>
__device__ __forceinline__ void issue_stage(const PagedAttnParams& p, uint8_t* stage, const StagePages& g, int h,
                                            int base, int end, int me) {
  constexpr int kCols = D / 16;
  const uint32_t dst = smem_u32(stage);
  const int P = p.c.P;
#pragma unroll
  for (int grp = 0; grp < 2; ++grp) {
    const int page = grp ? g.p1 : g.p0;
    const int64_t row = ((int64_t)max(page, 0) * p.c.Hkv + h) * P + (page >= 0 ? (grp ? g.o1 : g.o0) : 0);
    const uint8_t* k = p.c.k + row * D;
    const uint8_t* v = p.c.v + row * D;
    const int live = page >= 0 ? end - base - grp * 16 : 0;
#pragma unroll
    for (int x = 0; x < (16 * kCols + N - 1) / N; ++x) {
      const int i = me + x * N, r = i / kCols, c = i % kCols;
      if (16 * kCols % N != 0 && i >= 16 * kCols) break;
      const int bytes = r < live ? 16 : 0;
      const int off = r < live ? r * D + c * 16 : 0;
      const int at = (grp * 16 + r) * D + swz<D>(grp * 16 + r, c) * 16;
      cp_async16(dst + at, k + off, bytes);
      cp_async16(dst + kStageTokens * D + at, v + off, bytes);
    }
  }
  if (me < 4) {  // the scales: ks of both groups, then vs
    const int page = me & 1 ? g.p1 : g.p0;
    const float* src = (me & 2 ? p.c.vs : p.c.ks) + (int64_t)max(page, 0) * p.c.Hkv + h;
    cp_async4(dst + kStageTokens * D * 2 + me * 4, src, page >= 0 ? 4 : 0);
  }
  if (me == 0) {  // tokens of each group that are there
    int* f = reinterpret_cast<int*>(stage + kStageTokens * D * 2 + 16);
    f[0] = g.p0 >= 0 ? min(max(end - base, 0), 16) : 0;
    f[1] = g.p1 >= 0 ? min(max(end - base - 16, 0), 16) : 0;
  }
}

// A warp's rows: MT tiles of 16; this lane's are g and g + 8 of each (g = lane / 4).
template <int D, int MT>
struct Rows {
  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2], rf[MT][2];
  int pos[MT][2];     // position, or -1 for a row that is not there
  uint32_t ref;       // exponent field of the value scales' reference
  int pos_min, pos_max;  // of the warp's rows that are there

  __device__ __forceinline__ void clear() {
    ref = 1;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
  }
};

// Fragments of 16 query rows in shared memory: for each k-step and lane the four registers of the A operand.
// The lane holding row g reads channels 16 t + 4 s .. + 3 (and 64 more for the upper half of D = 128) of rows g
// and g + 8; every warp gets its rows' factors, those with `write` store the fragments.
template <int D>
__device__ __forceinline__ void load_q_tile(const PagedAttnParams& p, uint4* frag, int t0, int h, int row_first,
                                            int rows, float* rf, bool write) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool half = p.half != 0;
  uint32_t a[2][D / 16][2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row_first + g + 8 * r;
    const bool there = row < rows;
    const int tok = there ? row / p.G : 0, head = there ? row % p.G : 0;
    const uint16_t* src = p.q + (int64_t)(t0 + tok) * p.q_stride + (int64_t)(h * p.G + head) * D + 16 * t;
    float x[D / 64][16];
    float amax = 0.f;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      uint4 u = make_uint4(0, 0, 0, 0), w = u;
      if (there) {
        u = __ldg(reinterpret_cast<const uint4*>(src + 64 * hh));
        w = __ldg(reinterpret_cast<const uint4*>(src + 64 * hh) + 1);
      }
      const uint32_t z[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[hh][2 * i] = in_lo(z[i], half);
        x[hh][2 * i + 1] = in_hi(z[i], half);
        amax = fmaxf(amax, fmaxf(fabsf(x[hh][2 * i]), fabsf(x[hh][2 * i + 1])));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t e = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
    const float inv = pow2_of(254u - e);
    rf[r] = pow2_of(e) * p.scale;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const float* y = x[s >> 2] + 4 * (s & 3);
      a[r][s][0] = pack_half(y[0] * inv, y[1] * inv);
      a[r][s][1] = pack_half(y[2] * inv, y[3] * inv);
    }
  }
  if (!write) return;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) frag[s * 32 + lane] = make_uint4(a[0][s][0], a[1][s][0], a[0][s][1], a[1][s][1]);
}

template <int D, int MT>
__device__ __forceinline__ void set_rows(const PagedAttnParams& p, Rows<D, MT>& R, int row_first, int rows, int pos0) {
  const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row_first + 16 * t + g + 8 * r;
      R.pos[t][r] = row < rows ? pos0 + row / p.G : -1;
    }
  R.pos_min = row_first < rows ? pos0 + row_first / p.G : 0;
  R.pos_max = row_first < rows ? pos0 + (min(rows, row_first + 16 * MT) - 1) / p.G : -1;
}

// One stage of 32 tokens for the warp's rows.
template <int D, bool INT8, int MT>
__device__ __forceinline__ void do_stage(const PagedAttnParams& p, const uint8_t* stage, const uint4* qf,
                                         Rows<D, MT>& R, int base, int end) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float4 sc = *reinterpret_cast<const float4*>(stage + kStageTokens * D * 2);
  const int2 live = *reinterpret_cast<const int2*>(stage + kStageTokens * D * 2 + 16);
  float s[MT][4][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][j][e] = 0.f;
  // S = Q C_k^T: token tile j, lane (g, t) holds token 8 j + g, columns t and t + 4 of 16 codes
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = 8 * j + g;
    const uint8_t* src = stage + row * D;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      const uint4 c = *reinterpret_cast<const uint4*>(src + swz<D>(row, t + 4 * hh) * 16);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t b0, b1;
        codes_f16<INT8>(w[k], b0, b1);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint4 q = qf[(i * (D / 16) + hh * 4 + k) * 32 + lane];
          const uint32_t a[4] = {q.x, q.y, q.z, q.w};
          mma_f16(s[i][j], a, b0, b1);
        }
      }
    }
  }
  // A stage that every row sees whole needs no mask.
  const bool whole = live.x == 16 && live.y == 16 && base + kStageTokens <= R.pos_min + 1 &&
                     (p.W == 0 || base > R.pos_max - p.W || base + kStageTokens <= p.S);
  const uint32_t ref = max(R.ref, max(pow2_above(sc.z), pow2_above(sc.w)));
  const float down = pow2_of(R.ref) * pow2_of(254u - ref);
  const float v0 = sc.z * pow2_of(254u - ref), v1 = sc.w * pow2_of(254u - ref);
  bool moved = ref != R.ref;
  R.ref = ref;
  float corr[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float f0 = sc.x * R.rf[i][r], f1 = sc.y * R.rf[i][r];
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float z = s[i][j][2 * r + e] * (j < 2 ? f0 : f1);
          if (!whole) {
            const int in = 8 * (j & 1) + 2 * t + e;  // place within the group of 16
            const int tok = base + 16 * (j >> 1) + in;
            const bool seen = in < (j < 2 ? live.x : live.y) && tok <= R.pos[i][r] &&
                              (p.W == 0 || tok > R.pos[i][r] - p.W || tok < p.S);
            z = seen ? z : -INFINITY;
          }
          s[i][j][2 * r + e] = z;
          top = fmaxf(top, z);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m = fmaxf(R.m[i][r], top);
      const float shift = m == -INFINITY ? 0.f : m - 15.f;  // no token seen yet: every weight is 2^-inf
      corr[i][r] = exp2_fast(R.m[i][r] - (m == -INFINITY ? 0.f : m));
      moved |= m != R.m[i][r];
      R.m[i][r] = m;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w = exp2_fast(s[i][j][2 * r + e] - shift);
          sum += w;
          s[i][j][2 * r + e] = w * (j < 2 ? v0 : v1);
        }
      R.l[i][r] = R.l[i][r] * corr[i][r] + sum;
    }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const float c0 = corr[i][0] * down, c1 = corr[i][1] * down;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        R.o[i][j][0] *= c0;
        R.o[i][j][1] *= c0;
        R.o[i][j][2] *= c1;
        R.o[i][j][3] *= c1;
      }
    }
  }
  // O += P C_v: 16 tokens at a time; the lane holds channels g D/8 .. of tokens 2t, 2t + 1, 2t + 8, 2t + 9, and
  // product j covers channel j of every lane group
  const uint8_t* vst = stage + kStageTokens * D;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t a[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      a[i][0] = pack_half(s[i][2 * u][0], s[i][2 * u][1]);
      a[i][1] = pack_half(s[i][2 * u][2], s[i][2 * u][3]);
      a[i][2] = pack_half(s[i][2 * u + 1][0], s[i][2 * u + 1][1]);
      a[i][3] = pack_half(s[i][2 * u + 1][2], s[i][2 * u + 1][3]);
    }
    uint32_t c[4][D / 32];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = 16 * u + 2 * t + (x & 1) + 8 * (x >> 1);
      if (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4*>(vst + row * D + swz<D>(row, g) * 16);
        c[x][0] = w.x, c[x][1] = w.y, c[x][D / 32 - 2] = w.z, c[x][D / 32 - 1] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(vst + row * D + swz<D>(row, g >> 1) * 16 + (g & 1) * 8);
        c[x][0] = w.x, c[x][1] = w.y;
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t sel = hf ? 0x7362 : 0x5140;
        uint32_t b0[2], b1[2];
        codes_f16<INT8>(__byte_perm(c[0][w], c[1][w], sel), b0[0], b0[1]);
        codes_f16<INT8>(__byte_perm(c[2][w], c[3][w], sel), b1[0], b1[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < MT; ++i) mma_f16(R.o[i][w * 4 + hf * 2 + x], a[i], b0[x], b1[x]);
      }
  }
}

// Completes a row's sums over the four lanes that share it.
template <int D, int MT>
__device__ __forceinline__ void finish_sums(Rows<D, MT>& R) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l = R.l[i][r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      R.l[i][r] = l;
    }
}

// ---- the narrow form: up to 32 rows a KV head -----------------------------------------------------
//
// Bound by the codes' bytes.  The stages of all (sequence, KV head) units form one
// line that n_cta CTAs cut into equal parts, so ragged batches keep every SM busy
// to the end; the four warps of a CTA take its stages in turn, each through a ring
// of its own (no barrier in the loop), and are joined at each unit's end.  A unit
// that more than one CTA worked on is joined by paged_join_kernel.

__device__ __forceinline__ Span seq_span(const PagedAttnParams& p, const Seq& s) {
  const int pos0 = s.len - s.n;
  if (s.n == 0) return Span{0, 0, 0, 0, 0};
  return make_span(max(pos0, 0), s.len - 1, p.W, p.S);
}

// Stages of a sequence (for one KV head).
__device__ __forceinline__ int seq_stages(const PagedAttnParams& p, int b) {
  bool bad;
  const Seq s = read_seq(p.b, b, p.c.P, &bad);
  return seq_span(p, s).stages;
}
// All lanes: the stages of all units.
__device__ __forceinline__ int64_t line_total(const PagedAttnParams& p) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int b = lane; b < p.b.B; b += 32) sum += seq_stages(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * p.c.Hkv;
}
// All lanes: the sequence that stage x of the line lies in, and the line's stage
// at which its first unit begins.
__device__ __forceinline__ int line_find(const PagedAttnParams& p, int64_t x, int64_t& begin) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.b.B; b0 += 32) {
    int64_t mine = b0 + lane < p.b.B ? (int64_t)seq_stages(p, b0 + lane) * p.c.Hkv : 0;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > x);
    if (past) {
      const int l = __ffs(past) - 1;
      begin = __shfl_sync(0xffffffffu, before + upto - mine, l);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  begin = before;
  return p.b.B;
}
__device__ __forceinline__ int64_t cut(int64_t total, int n, int c) { return total * c / n; }

__device__ __forceinline__ void store_row(const PagedAttnParams& p, int64_t tok, int head, float lse2) {
  if (p.lse != nullptr) p.lse[tok * p.Hq + head] = lse2;
}

constexpr float kLn2 = 0.6931471805599453f;
// Natural logarithm of the sum whose weights are 2^(z - m + 15).
__device__ __forceinline__ float lse_of(float m, float l) { return m == -INFINITY ? -INFINITY : (m - 15.f + log2f(l)) * kLn2; }

template <int D, bool INT8, int MT>
__global__ void __launch_bounds__(kWarps * 32, NarrowGeo<D, MT>::kCtas) paged_narrow_kernel(const PagedAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kRing = NarrowGeo<D, MT>::kStages, kBytes = StageGeo<D>::kBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kRing * kBytes;
  uint4* qf = reinterpret_cast<uint4*>(smem + kWarps * kRing * kBytes);
  const uint32_t magic = (uint32_t)(((1ull << 32) + p.c.P / 16 - 1) / (uint32_t)(p.c.P / 16));

  const int64_t total = line_total(p);
  const int64_t first = cut(total, p.n_cta, blockIdx.x), last = cut(total, p.n_cta, blockIdx.x + 1);
  int64_t at = first;
  pdl_allow_dependents();  // the join may take its place; it waits for this grid's end
  while (at < last) {
    // the unit that stage `at` lies in, and the part of it that is this CTA's
    int64_t begin;
    const int b = line_find(p, at, begin);
    bool bad;
    const Seq seq = read_seq(p.b, b, p.c.P, &bad);
    const Span span = seq_span(p, seq);
    const int h = (int)((at - begin) / span.stages);
    const int64_t ubegin = begin + (int64_t)h * span.stages;
    const int s0 = (int)(at - ubegin), s1 = (int)min((int64_t)span.stages, last - ubegin);
    const bool complete = s0 == 0 && s1 == span.stages;
    const int slot = 2 * blockIdx.x + (at == first ? 0 : 1);
    at = ubegin + s1;
    const int rows = min(seq.n * p.G, 16 * MT), pos0 = seq.len - seq.n;
    const int32_t* table = p.b.table + (int64_t)b * p.b.mp;
    if (bad && h == 0 && s0 == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);

    // start the first stages, then the queries
    const int mine = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;
    StagePages nxt;
    int base, end;
    auto find = [&](int i) {
      stage_range(span, s0 + warp + i * kWarps, base, end);
      nxt = stage_pages(p, table, base, end, magic);
    };
    if (mine > 0) find(0);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
      if (i < mine) {
        issue_stage<D, 32>(p, ring + i * kBytes, nxt, h, base, end, lane);
        if (i + 1 < mine) find(i + 1);
      }
      cp_commit();
    }
    Rows<D, MT> R;
    R.clear();
    set_rows<D, MT>(p, R, 0, rows, pos0);
#pragma unroll
    for (int i = 0; i < MT; ++i) load_q_tile<D>(p, qf + i * (D / 16) * 32, seq.t0, h, 16 * i, rows, R.rf[i], warp == i);
    __syncthreads();

    int slot_in = kRing - 1, slot_out = 0;
    for (int i = 0; i < mine; ++i) {
      cp_wait<kRing - 2>();
      __syncwarp();
      if (i + kRing - 1 < mine) {
        issue_stage<D, 32>(p, ring + slot_in * kBytes, nxt, h, base, end, lane);
        if (i + kRing < mine) find(i + kRing);
      }
      cp_commit();
      int sb, se;
      stage_range(span, s0 + warp + i * kWarps, sb, se);
      do_stage<D, INT8, MT>(p, ring + slot_out * kBytes, qf, R, sb, se);
      __syncwarp();
      slot_in = slot_in + 1 == kRing ? 0 : slot_in + 1;
      slot_out = slot_out + 1 == kRing ? 0 : slot_out + 1;
    }
    cp_wait<0>();
    finish_sums<D, MT>(R);

    // Join the warps: sums and maxima first, then the outputs, through the rings' memory.
    __syncthreads();
    float* head = reinterpret_cast<float*>(qf);  // [warp][row][m, l, ref]
    float* body = reinterpret_cast<float*>(smem);  // [warp][row][D]
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * i + g + 8 * r;
        if (t == 0) {
          float* e = head + (warp * 16 * MT + row) * 3;
          e[0] = R.m[i][r], e[1] = R.l[i][r], e[2] = pow2_of(R.ref);
        }
        // lane (g, t) holds channels 2 t and 2 t + 1 of the 8 lane groups: product j's columns are channel j of group 2 t
        float* o = body + (warp * 16 * MT + row) * D;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[(2 * t) * (D / 8) + j] = R.o[i][j][2 * r];
          o[(2 * t + 1) * (D / 8) + j] = R.o[i][j][2 * r + 1];
        }
      }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
      const int row = x / (D / 4), c = x % (D / 4) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, head[(w * 16 * MT + row) * 3]);
      float l = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* e = head + (w * 16 * MT + row) * 3;
        f[w] = m == -INFINITY ? 0.f : exp2f(e[0] - m);
        l += e[1] * f[w];
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(body + (w * 16 * MT + row) * D + c);
        const float k = f[w] * inv * head[(w * 16 * MT + row) * 3 + 2];
        y.x += o.x * k, y.y += o.y * k, y.z += o.z * k, y.w += o.w * k;
      }
      const int64_t tok = seq.t0 + row / p.G;
      const int hd = h * p.G + row % p.G;
      if (complete) {
        *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + (int64_t)hd * D + c) =
            make_uint2(pack_out(y.x, y.y, p.half), pack_out(y.z, y.w, p.half));
        if (c == 0) store_row(p, tok, hd, lse_of(m, l));
      } else {
        float* ws = p.ws + ((int64_t)slot * 16 * MT + row) * (D + 4);
        *reinterpret_cast<float4*>(ws + c) = y;
        if (c == 0) ws[D] = m, ws[D + 1] = l;
      }
    }
    __syncthreads();
  }
}

// Joins n parts of a row: `part(i)` is the i-th part's [D outputs, m, l].  kJoinThreads threads; returns the four
// channels 4 c .. of thread c < D / 4, the row's maximum and sum.
constexpr int kJoinThreads = 128;
constexpr int kJoinMost = 512;  // parts

template <int D, class F>
__device__ __forceinline__ float4 join_parts(int n, F part, float& top, float& sum) {
  __shared__ float weight[kJoinMost], red[2][kJoinThreads / 32];
  __shared__ float4 acc[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  float m = -INFINITY;
  for (int i = tid; i < n; i += kJoinThreads) m = fmaxf(m, part(i)[D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.f;
  for (int i = tid; i < n; i += kJoinThreads) {
    const float* e = part(i);
    const float w = m == -INFINITY ? 0.f : exp2f(e[D] - m) * e[D + 1];
    weight[i] = w;
    l += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[1][tid >> 5] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) l += red[1][w];
  // D / 4 threads a part
  constexpr int kSide = kJoinThreads / (D / 4);
  const int c = tid % (D / 4), first = tid / (D / 4);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = first; i < n; i += kSide) {
    const float w = weight[i];
    const float4 o = *reinterpret_cast<const float4*>(part(i) + 4 * c);
    y.x += w * o.x, y.y += w * o.y, y.z += w * o.z, y.w += w * o.w;
  }
  acc[tid] = y;
  __syncthreads();
  const float inv = l == 0.f ? 0.f : 1.f / l;
  y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int g = 0; g < kSide; ++g) {
    const float4 o = acc[g * (D / 4) + c];
    y.x += o.x, y.y += o.y, y.z += o.z, y.w += o.w;
  }
  y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
  top = m;
  sum = l;
  return y;
}

__device__ __forceinline__ void store_joined(const PagedAttnParams& p, int64_t tok, int hd, int D, int c, const float4& y,
                                             float m, float l) {
  *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + (int64_t)hd * D + 4 * c) =
      make_uint2(pack_out(y.x, y.y, p.half), pack_out(y.z, y.w, p.half));
  if (c == 0) store_row(p, tok, hd, lse_of(m, l));
}

// Joins the parts of units that more than one CTA worked on, and writes the rows
// of units with no visible token.  One CTA a (unit, row).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedAttnParams p, int tile_rows) {
  const int unit = blockIdx.x, row = blockIdx.y;
  const int b = unit / p.c.Hkv, h = unit % p.c.Hkv;
  bool bad;
  const Seq seq = read_seq(p.b, b, p.c.P, &bad);
  if (row >= min(seq.n * p.G, tile_rows)) {
    pdl_wait_primary();  // every block: this grid's end stands for the attention's too
    return;
  }
  const int64_t tok = seq.t0 + row / p.G;
  const int hd = h * p.G + row % p.G;
  const int stages = seq_span(p, seq).stages;
  if (stages == 0) {
    pdl_wait_primary();
    if (threadIdx.x < D / 4) store_joined(p, tok, hd, D, threadIdx.x, make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
    return;
  }
  // the line up to this sequence
  const int lane = threadIdx.x & 31;
  int64_t before = 0, total = 0;
  for (int i = lane; i < p.b.B; i += 32) {
    const int64_t n = seq_stages(p, i);
    total += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total *= p.c.Hkv;
  const int64_t begin = before * p.c.Hkv + (int64_t)h * stages, endu = begin + stages;
  // the CTA whose part [total c / n, total (c + 1) / n) holds a stage x is c = ceil((x + 1) n / total) - 1;
  // with fewer stages than CTAs the parts are of one stage or none, and those in between that have none are passed over
  const int c0 = (int)(((begin + 1) * p.n_cta + total - 1) / total) - 1;
  const int c1 = (int)((endu * p.n_cta + total - 1) / total) - 1;
  pdl_wait_primary();
  if (c0 == c1) return;  // complete in one CTA
  const bool sparse = total < p.n_cta;
  const int n = sparse ? stages : c1 - c0 + 1;
  const bool starts_before = cut(total, p.n_cta, c0) < begin;
  auto part = [&](int i) -> const float* {
    const int c = sparse ? (int)(((begin + i + 1) * p.n_cta + total - 1) / total) - 1 : c0 + i;
    const int64_t slot = 2 * (int64_t)c + (i == 0 && starts_before ? 1 : 0);
    return p.ws + (slot * tile_rows + row) * (D + 4);
  };
  float m, l;
  const float4 y = join_parts<D>(n, part, m, l);
  if (threadIdx.x < D / 4) store_joined(p, tok, hd, D, threadIdx.x, y, m, l);
}

// ---- the wide form: many rows a KV head --------------------------------------------------------------
//
// A CTA takes 128 rows, 32 a warp, and passes the stages its rows can see through
// one shared ring; every warp converts the codes itself (the conversions run
// beside the other warps' products).  Few row tiles over a long cache are cut
// into n_splits parts of their stages, joined by paged_join_rows_kernel.

constexpr int kWideRing = 4;

template <int D, bool INT8>
__global__ void __launch_bounds__(kWarps * 32, kWideCtasPerSm) paged_wide_kernel(const PagedAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int MT = 2, kBytes = StageGeo<D>::kBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint4* qf = reinterpret_cast<uint4*>(smem + kWideRing * kBytes);
  const uint32_t magic = (uint32_t)(((1ull << 32) + p.c.P / 16 - 1) / (uint32_t)(p.c.P / 16));
  const int unit = blockIdx.y, b = unit / p.c.Hkv, h = unit % p.c.Hkv;
  // the tiles that see most come first
  const int tile = (int)(gridDim.x / p.n_splits) - 1 - (int)(blockIdx.x / p.n_splits);
  const int split = blockIdx.x % p.n_splits;
  bool bad;
  const Seq seq = read_seq(p.b, b, p.c.P, &bad);
  if (bad && h == 0 && tile == 0 && split == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
  const int rows = seq.n * p.G, row0 = tile * kWideRows, pos0 = seq.len - seq.n;
  if (row0 >= rows) return;
  const int pos_min = pos0 + row0 / p.G, pos_max = pos0 + (min(rows, row0 + kWideRows) - 1) / p.G;
  const Span span = pos_max >= 0 ? make_span(max(pos_min, 0), pos_max, p.W, p.S) : Span{0, 0, 0, 0, 0};
  const int s0 = (int)((int64_t)span.stages * split / p.n_splits);
  const int s1 = (int)((int64_t)span.stages * (split + 1) / p.n_splits);
  const int32_t* table = p.b.table + (int64_t)b * p.b.mp;

  StagePages nxt;
  int base, end;
  auto find = [&](int i) {
    stage_range(span, i, base, end);
    nxt = stage_pages(p, table, base, end, magic);
  };
  if (s0 < s1) find(s0);
#pragma unroll
  for (int i = 0; i < kWideRing - 1; ++i) {
    if (s0 + i < s1) {
      issue_stage<D, kWarps * 32>(p, smem + i * kBytes, nxt, h, base, end, threadIdx.x);
      if (s0 + i + 1 < s1) find(s0 + i + 1);
    }
    cp_commit();
  }
  Rows<D, MT> R;
  R.clear();
  set_rows<D, MT>(p, R, row0 + 32 * warp, rows, pos0);
  uint4* my = qf + warp * MT * (D / 16) * 32;
#pragma unroll
  for (int i = 0; i < MT; ++i) load_q_tile<D>(p, my + i * (D / 16) * 32, seq.t0, h, row0 + 32 * warp + 16 * i, rows, R.rf[i], true);
  for (int i = s0; i < s1; ++i) {
    cp_wait<kWideRing - 2>();
    __syncthreads();  // the stage is there, and everyone is done with the one before
    if (i + kWideRing - 1 < s1) {
      issue_stage<D, kWarps * 32>(p, smem + (i - s0 + kWideRing - 1) % kWideRing * kBytes, nxt, h, base, end,
                                  threadIdx.x);
      if (i + kWideRing < s1) find(i + kWideRing);
    }
    cp_commit();
    int sb, se;
    stage_range(span, i, sb, se);
    if (sb <= R.pos_max) do_stage<D, INT8, MT>(p, smem + (i - s0) % kWideRing * kBytes, my, R, sb, se);
  }
  cp_wait<0>();
  finish_sums<D, MT>(R);
  // Rows leave through shared memory, a warp's 16 at a time, so that they are stored in their own order.
  __syncthreads();
  float* body = reinterpret_cast<float*>(smem) + warp * 16 * (D + 4);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float inv = R.l[i][r] == 0.f ? 0.f : pow2_of(R.ref) / R.l[i][r];
      float* o = body + (g + 8 * r) * (D + 4);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[(2 * t) * (D / 8) + j] = R.o[i][j][2 * r] * inv;
        o[(2 * t + 1) * (D / 8) + j] = R.o[i][j][2 * r + 1] * inv;
      }
      if (t == 0) o[D] = R.m[i][r], o[D + 1] = R.l[i][r];
    }
    __syncwarp();
    const int first = row0 + 32 * warp + 16 * i;
    for (int x = lane; x < 16 * (D / 4); x += 32) {
      const int rr = x / (D / 4), c = x % (D / 4) * 4, row = first + rr;
      if (row >= rows) break;
      const float4 y = *reinterpret_cast<const float4*>(body + rr * (D + 4) + c);
      const float m = body[rr * (D + 4) + D], l = body[rr * (D + 4) + D + 1];
      const int64_t tok = seq.t0 + row / p.G;
      const int hd = h * p.G + row % p.G;
      if (p.n_splits == 1) {
        *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + (int64_t)hd * D + c) =
            make_uint2(pack_out(y.x, y.y, p.half), pack_out(y.z, y.w, p.half));
        if (c == 0) store_row(p, tok, hd, lse_of(m, l));
      } else {
        float* ws = p.ws + (((int64_t)split * p.b.n_new + tok) * p.Hq + hd) * (D + 4);
        *reinterpret_cast<float4*>(ws + c) = y;
        if (c == 0) ws[D] = m, ws[D + 1] = l;
      }
    }
    __syncwarp();
  }
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_rows_kernel(const PagedAttnParams p) {
  bool bad;
  const Seq seq = read_seq(p.b, blockIdx.z, p.c.P, &bad);
  pdl_wait_primary();
  if ((int)blockIdx.y >= seq.n) return;
  const int64_t tok = seq.t0 + blockIdx.y;
  const int hd = blockIdx.x;
  auto part = [&](int i) -> const float* { return p.ws + (((int64_t)i * p.b.n_new + tok) * p.Hq + hd) * (D + 4); };
  float m, l;
  const float4 y = join_parts<D>(p.n_splits, part, m, l);
  if (threadIdx.x < D / 4) store_joined(p, tok, hd, D, threadIdx.x, y, m, l);
}

// ---- launches -----------------------------------------------------------------------------------------
template <class... A>
cudaError_t launch(void (*f)(A...), dim3 grid, dim3 block, size_t smem, bool chained, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = chained ? 1 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&c, f, args...);
}

template <int D, bool INT8, int MT>
cudaError_t narrow(const PagedAttnParams& p, cudaStream_t s) {
  constexpr size_t rings = (size_t)kWarps * NarrowGeo<D, MT>::kStages * StageGeo<D>::kBytes;
  constexpr size_t frags = (size_t)MT * (D / 16) * 32 * sizeof(uint4);
  static_assert(rings >= (size_t)kWarps * 16 * MT * D * sizeof(float), "the join's rows fit the rings");
  static_assert(frags >= (size_t)kWarps * 16 * MT * 3 * sizeof(float), "the join's sums fit the fragments");
  cudaError_t e = launch(paged_narrow_kernel<D, INT8, MT>, dim3(p.n_cta), dim3(kWarps * 32), rings + frags, false, s, p);
  if (e != cudaSuccess) return e;
  const int rows = p.b.max_new * p.G < 16 * MT ? p.b.max_new * p.G : 16 * MT;
  return launch(paged_join_kernel<D>, dim3(p.b.B * p.c.Hkv, rows), dim3(kJoinThreads), 0, true, s, p, 16 * MT);
}

template <int D, bool INT8>
cudaError_t wide(const PagedAttnParams& p, cudaStream_t s) {
  constexpr size_t ring = (size_t)kWideRing * StageGeo<D>::kBytes;
  constexpr size_t frags = (size_t)kWarps * 2 * (D / 16) * 32 * sizeof(uint4);
  constexpr size_t out = (size_t)kWarps * 16 * (D + 4) * sizeof(float);
  constexpr size_t smem = ring + frags > out ? ring + frags : out;
  const int64_t tiles = ((int64_t)p.b.max_new * p.G + kWideRows - 1) / kWideRows;
  cudaError_t e = launch(paged_wide_kernel<D, INT8>, dim3((unsigned)(tiles * p.n_splits), p.b.B * p.c.Hkv),
                         dim3(kWarps * 32), smem, false, s, p);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  return launch(paged_join_rows_kernel<D>, dim3(p.Hq, p.b.max_new, p.b.B), dim3(kJoinThreads), 0, true, s, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  const int lanes = p.D / 16;
  int threads = (p.c.P * lanes / kAppendRows + 31) / 32 * 32;
  const int64_t q_threads = p.q != nullptr ? (int64_t)p.b.n_new * ((p.Hq + 3) / 4) * lanes : 0;
  const int64_t blocks = p.kv_blocks + (q_threads + threads - 1) / threads;
  return launch(p.interleaved ? paged_append_kernel<true> : paged_append_kernel<false>, dim3((unsigned)blocks),
                dim3(threads), 0, false, s, p);
}

cudaError_t launch_paged_narrow(const PagedAttnParams& p, int D, int int8, int tiles, cudaStream_t s) {
  if (D == 128)
    return int8 ? (tiles == 1 ? narrow<128, true, 1>(p, s) : narrow<128, true, 2>(p, s))
                : (tiles == 1 ? narrow<128, false, 1>(p, s) : narrow<128, false, 2>(p, s));
  return int8 ? (tiles == 1 ? narrow<64, true, 1>(p, s) : narrow<64, true, 2>(p, s))
              : (tiles == 1 ? narrow<64, false, 1>(p, s) : narrow<64, false, 2>(p, s));
}

cudaError_t launch_paged_wide(const PagedAttnParams& p, int D, int int8, cudaStream_t s) {
  if (D == 128) return int8 ? wide<128, true>(p, s) : wide<128, false>(p, s);
  return int8 ? wide<64, true>(p, s) : wide<64, false>(p, s);
}

}  // namespace hyb
