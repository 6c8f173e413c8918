// Append of a step's tokens to the paged 8-bit cache, keys and queries rotated.
#include "k_paged.cuh"

namespace hyb {
namespace {

// One CTA takes the new tokens that fall into one page of one sequence, for one
// KV head and for keys or values: it holds them rotated in registers (4 rows of
// 16 channels a thread), reduces their largest magnitude, settles the page's
// scale, rewrites the codes that the page already holds if the scale grew, and
// writes the new codes.  So each input is read once and each code written once.
// CTAs behind those rotate the queries, a thread 16 channels of four heads with one set of angles.
//
// Bound by bytes for a prompt, by the chain page table -> row -> scale for a few tokens.  32768 tokens of 32 and 8 heads of
// 128: 150 us, 5.0 TB/s (of the copies' 6.6); 2 rows a thread 194 us against 171 for 4 when measured.  8 sequences, one
// token: 5.3 us.  Queries in a launch of their own take longer at all sizes: 2048 tokens 15.0 us against 11.1, 32768 152
// against 150.

constexpr int kAppendRows = 4;  // rows a thread holds

// a * c - b * s, correctly rounded for 16-bit a and b but for ties within 2^-45:
// the products' rounding errors are exact (fma), their difference's too (two-sum).
__device__ __forceinline__ float diff_of_products(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float q = __fmul_rn(b, s), qe = __fmaf_rn(b, s, -q);
  const float d = __fsub_rn(p, q);
  const float bb = __fsub_rn(d, p);
  const float de = __fsub_rn(__fsub_rn(p, __fsub_rn(d, bb)), __fadd_rn(q, bb));
  return __fadd_rn(d, __fadd_rn(de, __fsub_rn(pe, qe)));  // NaN where an input is not finite, or a product overflows
}

template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
  // times 1 / 127, as a tensor divided by a number is computed: a unit in the last place would turn ties of codes
  if (INT8) return fmaxf(__fmul_rn(amax, 1.f / 127.f), 1.17549435e-38f);
  // the smallest power of two x in [2^-126, 2^126] with amax <= 448 x:
  // 448 = 1.75 * 2^8, so x = 2^(e - 8) or the next for amax = m 2^e, 1 <= m < 2
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, -126), 126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Code of y (already divided by the scale, not NaN): nearest, ties to even, saturating.
template <bool INT8>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  if (INT8) {
    const int a = __float2int_rn(fminf(fmaxf(lo, -127.f), 127.f));
    const int b = __float2int_rn(fminf(fmaxf(hi, -127.f), 127.f));
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8);
  }
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool INT8>
__device__ __forceinline__ uint32_t code4(const float* y, float inv) {
  return code2<INT8>(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv)) | (code2<INT8>(__fmul_rn(y[2], inv), __fmul_rn(y[3], inv)) << 16);
}
// The value a code stands for, without its scale (e4m3's NaN codes stay NaN).
template <bool INT8>
__device__ __forceinline__ float value_of(uint32_t byte) {
  if (INT8) return (float)(int)(int8_t)byte;
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
// The runs as they are loaded, and as values.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_runs(const uint16_t* row, const Runs& r) {
  return Raw{*reinterpret_cast<const uint4*>(row + r.c0), *reinterpret_cast<const uint4*>(row + r.c1)};
}
__device__ __forceinline__ void to_values(const Raw& raw, bool half, float* x) {
  const uint32_t w[8] = {raw.a.x, raw.a.y, raw.a.z, raw.a.w, raw.b.x, raw.b.y, raw.b.z, raw.b.w};
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
  const float4 x = c[0], y = c[1], z = s[0], w = s[1];
  a.c[0] = x.x, a.c[1] = x.y, a.c[2] = x.z, a.c[3] = x.w, a.c[4] = y.x, a.c[5] = y.y, a.c[6] = y.z, a.c[7] = y.w;
  a.s[0] = z.x, a.s[1] = z.y, a.s[2] = z.z, a.s[3] = z.w, a.s[4] = w.x, a.s[5] = w.y, a.s[6] = w.z, a.s[7] = w.w;
}
enum TurnAs { kExact, kPlain, kNear };
template <TurnAs HOW>
__device__ __forceinline__ void turn(float* x, const Angles& a, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& u = interleaved ? x[2 * i] : x[i];
    float& w = interleaved ? x[2 * i + 1] : x[8 + i];
    const float p = u, q = w;
    if (HOW == kExact) {
      u = diff_of_products(p, a.c[i], q, a.s[i]);
      w = diff_of_products(q, a.c[i], -p, a.s[i]);
    } else if (HOW == kPlain) {
      u = p * a.c[i] - q * a.s[i];
      w = q * a.c[i] + p * a.s[i];
    } else {  // an output of 16 bits: one rounding of a product's error is enough
      const float m = __fmul_rn(q, a.s[i]), n = __fmul_rn(p, a.s[i]);
      u = __fsub_rn(__fmaf_rn(p, a.c[i], -m), __fmaf_rn(q, a.s[i], -m));
      w = __fadd_rn(__fmaf_rn(q, a.c[i], n), __fmaf_rn(p, a.s[i], -n));
    }
  }
}

// The query part: thread `at` turns the same channels of 4 heads of one token.
template <bool INTERLEAVED, bool HALF>
__device__ __forceinline__ void rotate_queries(const PagedAppendParams& p, int64_t at) {
  constexpr bool half = HALF;
  const int lanes = p.D / 16, P = p.c.P;
  const int groups = (p.Hq + 3) / 4;
  const int j = (int)(at % lanes);
  const int64_t rest = at / lanes;
  const int hg = (int)(rest % groups);
  const int64_t t = rest / groups;
  if (t >= p.b.n_new) return;
  const Runs r = lane_runs(j, p.rot, INTERLEAVED);
  const int heads = min(4, p.Hq - hg * 4);
  Raw raw[4];  // under way before the token's sequence is known
#pragma unroll
  for (int h = 0; h < 4; ++h)
    if (h < heads) raw[h] = load_runs(p.q + t * p.q_stride + (int64_t)(hg * 4 + h) * p.D, r);
  // the token's sequence: the last b with cu[b] <= t
  int lo = 0, hi = p.b.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.b.cu[mid] <= t) lo = mid; else hi = mid;
  }
  bool bad;
  const Seq s = read_seq(p.b, lo, P, &bad);
  if (t < s.t0 || t >= s.t0 + s.n) return;  // a row behind the last sequence
  Angles a;
  if (r.angle >= 0) {
    const int pos = s.pos0 + (int)(t - s.t0);
    if (pos < 0 || pos >= p.n_pos) raise(p.status, HYB_STATUS_BAD_LENGTH);
    load_angles(a, p.rope + (int64_t)min(max(pos, 0), p.n_pos - 1) * p.rot, p.rot, r.angle);
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (h >= heads) break;
    float x[16];
    to_values(raw[h], half, x);
    if (r.angle >= 0) turn<kNear>(x, a, INTERLEAVED);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_out(x[2 * i], x[2 * i + 1], half);
    uint16_t* row = p.q_out + t * p.qo_stride + (int64_t)(hg * 4 + h) * p.D;
    *reinterpret_cast<uint4*>(row + r.c0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + r.c1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool INTERLEAVED, bool HALF, bool INT8>
__global__ void __launch_bounds__(512) paged_append_kernel(const PagedAppendParams p) {
  constexpr bool half = HALF;
  pdl_wait_primary();
  pdl_allow_dependents();
  const int lanes = p.D / 16;  // lanes of a row: 4 or 8
  const int P = p.c.P;

  if ((int64_t)blockIdx.x >= p.kv_blocks) {
    rotate_queries<INTERLEAVED, HALF>(p, ((int64_t)blockIdx.x - p.kv_blocks) * blockDim.x + threadIdx.x);
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
  const int start = s.pos0, first = max(start, 0);  // positions of the first new token, and of the first that has one
  const int pg = first / P + pi;                    // page of the sequence
  if (pg >= p.b.mp) return;                         // tokens past the table are skipped
  const int lo = max(pg * P, first), hi = min((pg + 1) * P, start + s.n);
  if (lo >= hi) return;
  const int j = threadIdx.x % lanes, row0 = threadIdx.x / lanes, step = blockDim.x / lanes;
  const Runs r = lane_runs(j, values ? 0 : p.rot, INTERLEAVED);
  const uint16_t* in = values ? p.v : p.k;
  const int64_t stride = values ? p.v_stride : p.k_stride;
  Raw raw[kAppendRows];  // under way before the page is known
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos < hi) raw[i] = load_runs(in + (int64_t)(s.t0 + pos - start) * stride + (int64_t)h * p.D, r);
  }
  const int page = p.b.table[(int64_t)b * p.b.mp + pg];
  if (page < 0 || page >= p.c.n_pages) {
    if (threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_PAGE);
    return;
  }
  float* scale_at = (values ? p.c.vs : p.c.ks) + (int64_t)page * p.c.Hkv + h;
  uint8_t* codes = (values ? p.c.v : p.c.k) + ((int64_t)page * p.c.Hkv + h) * P * p.D;
  const int older = lo - pg * P;  // tokens that the page held before
  const float was = older > 0 ? *scale_at : 0.f;

  float x[kAppendRows][16];
  uint32_t top = 0;  // the largest magnitude's bits, which order like it; past those of FLT_MAX where one is not finite
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos >= hi) continue;
    to_values(raw[i], half, x[i]);
    if (r.angle >= 0) {
      Angles a;
      if (pos >= p.n_pos) raise(p.status, HYB_STATUS_BAD_LENGTH);
      load_angles(a, p.rope + (int64_t)min(pos, p.n_pos - 1) * p.rot, p.rot, r.angle);
      turn<kExact>(x[i], a, INTERLEAVED);
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) top = max(top, __float_as_uint(x[i][c]) & 0x7fffffffu);
  }
  __shared__ uint32_t part[2][16];
  auto block_top = [&](uint32_t* shared) {
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = max(top, shared[w]);
  };
  block_top(part[0]);
  if (top >= 0x7f800000u) {
    // Some value is not finite.  Take the plain rotation where the exact one has no value, store NaN as 0, and leave
    // what is not finite out of the scale.
    bool odd = false;
    top = 0;
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
      const int pos = lo + row0 + i * step;
      if (pos >= hi) continue;
      float y[16];
      to_values(load_runs(in + (int64_t)(s.t0 + pos - start) * stride + (int64_t)h * p.D, r), half, y);
      if (r.angle >= 0) {
        Angles a;
        load_angles(a, p.rope + (int64_t)min(pos, p.n_pos - 1) * p.rot, p.rot, r.angle);
        turn<kPlain>(y, a, INTERLEAVED);
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (!isfinite(x[i][c])) x[i][c] = y[c];
        odd |= !isfinite(x[i][c]);
        if (isnan(x[i][c])) x[i][c] = 0.f;
        if (!isinf(x[i][c])) top = max(top, __float_as_uint(x[i][c]) & 0x7fffffffu);
      }
    }
    if (odd) raise(p.status, HYB_STATUS_NONFINITE);
    block_top(part[1]);
  }
  const float amax = __uint_as_float(top);
  const float need = scale_for<INT8>(amax);
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
      for (int i = 0; i < 4; ++i) y[i] = value_of<INT8>((c >> (8 * i)) & 0xffu);
      *at = code4<INT8>(y, ratio);
    }
  }
  if (threadIdx.x == 0 && !(older > 0 && now == was)) *scale_at = now;
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int pos = lo + row0 + i * step;
    if (pos >= hi) continue;
    uint8_t* row = codes + (int64_t)(pos - pg * P) * p.D;
    *reinterpret_cast<uint2*>(row + r.c0) = make_uint2(code4<INT8>(x[i], inv), code4<INT8>(x[i] + 4, inv));
    *reinterpret_cast<uint2*>(row + r.c1) = make_uint2(code4<INT8>(x[i] + 8, inv), code4<INT8>(x[i] + 12, inv));
  }
}

template <bool INTERLEAVED, bool HALF>
cudaError_t append(const PagedAppendParams& p, cudaStream_t s) {
  const int lanes = p.D / 16;
  const int threads = (p.c.P * lanes / kAppendRows + 31) / 32 * 32;
  const int64_t q_threads = p.q != nullptr ? (int64_t)p.b.n_new * ((p.Hq + 3) / 4) * lanes : 0;
  const int64_t blocks = p.kv_blocks + (q_threads + threads - 1) / threads;
  return launch(p.int8 ? paged_append_kernel<INTERLEAVED, HALF, true> : paged_append_kernel<INTERLEAVED, HALF, false>,
                dim3((unsigned)blocks), dim3(threads), 0, true, s, p);
}
}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  if (p.half) return p.interleaved ? append<true, true>(p, s) : append<false, true>(p, s);
  return p.interleaved ? append<true, false>(p, s) : append<false, false>(p, s);
}

}  // namespace hyb
