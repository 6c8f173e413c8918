// Device helpers shared by the kernels of the paged 8-bit cache.
//
// These kernels start before the one before them on the stream has ended (and wait for it before they read anything), so
// what they read may still be written while they run: plain loads only, none by the path of read-only data.
#pragma once

#include <cuda_fp16.h>

#include <cfloat>
#include <climits>

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
  int t0, n;  // first row, new tokens
  int pos0;   // position of the first row
  int cap;    // tokens that the page table has room for
};

// Reads a sequence's ranges and holds its rows within what the caller said: within [0, n_new), at most max_new of
// them.  A row keeps its position, lens - cu[i + 1] + row, whatever else is held: what falls outside [0, cap) is for the
// caller to skip.  Positions from pos0 to pos0 + n fit 32 bits (those below -2^30 are as good as -2^30, n being at most
// 2^30).
__device__ __forceinline__ Seq read_seq(const PagedBatch& b, int i, int P, bool* bad) {
  Seq s;
  const int c0 = b.cu[i], c1 = b.cu[i + 1], len = b.lens[i];
  s.t0 = min(max(c0, 0), b.n_new);
  const int t1 = min(max(c1, s.t0), b.n_new);
  s.n = min(t1 - s.t0, b.max_new);
  s.cap = b.mp * P;  // at most 2^30
  s.pos0 = (int)min(max((int64_t)len - c1 + s.t0, -((int64_t)1 << 30)), (int64_t)INT_MAX - s.n);
  const int64_t n = (int64_t)c1 - c0;
  *bad = s.t0 != c0 || s.n != n || len > s.cap || len < n;
  return s;
}

// ---- codes and scales ---------------------------------------------------------------------------
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
// 1 / x of a power of two x from 2^-126 to 2^126.
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// ---- what a row tile sees -------------------------------------------------------------------------
// Where the visible tokens of a row tile lie: sinks [0, sink), then [lo, hi)
// from a multiple of 16; stages of T tokens, the sinks' first.
template <int T>
struct Span {
  int sink, lo, hi, sink_stages, stages;
};
template <int T>
__device__ __forceinline__ Span<T> make_span(int pos_min, int pos_max, int cap, int W, int S) {
  Span<T> s;
  s.hi = min(pos_max + 1, cap);
  s.lo = W > 0 ? max(pos_min - W + 1, 0) & ~15 : 0;
  s.sink = W > 0 ? min(S, min(s.lo, s.hi)) : 0;  // positions past the table may have lo > hi
  s.sink_stages = (s.sink + T - 1) / T;
  s.stages = s.sink_stages + (max(s.hi - s.lo, 0) + T - 1) / T;
  return s;
}
// The first stage of a window begins at a multiple of 16: no row sees its tokens [gap, from).
struct Gap {
  int gap, from;
};
__device__ __forceinline__ Gap gap_of(const PagedAttnParams& p, int lo, int pos_min) {
  const int from = max(max(pos_min, 0) - p.W + 1, 0);
  return Gap{min(max(lo, p.S), from), from};
}
template <int T>
__device__ __forceinline__ void stage_range(const Span<T>& s, int st, int& base, int& end) {
  if (st < s.sink_stages) {
    base = st * T;
    end = min(base + T, s.sink);
  } else {
    base = s.lo + (st - s.sink_stages) * T;
    end = min(base + T, s.hi);
  }
}

// ---- the line of all stages -----------------------------------------------------------------------
//
// The stages of all (sequence, KV head) units, one after the other, cut into equal parts for the CTAs.

template <int T>
__device__ __forceinline__ Span<T> seq_span(const PagedAttnParams& p, const Seq& s) {
  if (s.n == 0 || s.pos0 + s.n <= 0) return Span<T>{0, 0, 0, 0, 0};
  return make_span<T>(max(s.pos0, 0), s.pos0 + s.n - 1, s.cap, p.W, p.S);
}

// The line's geometry, in all lanes of a warp.  Stage counts fit 31 bits (the host
// refuses more).
struct Line {
  uint32_t total;   // stages in all
  uint32_t per;     // of each CTA: a multiple of p.quantum
  uint32_t mine;    // lane's: stages of all units of sequence `lane`, and those before it
  uint32_t before;
};

// Stages of all of a sequence's units.  `tell`: what contradicts the caller's limits goes to the status.
template <int T>
__device__ __forceinline__ uint32_t seq_stages(const PagedAttnParams& p, int b, bool tell) {
  bool bad;
  const Seq s = read_seq(p.b, b, p.c.P, &bad);
  if (bad && tell) raise(p.status, HYB_STATUS_BAD_LENGTH);
  return (uint32_t)seq_span<T>(p, s).stages * (uint32_t)p.c.Hkv;
}
__device__ __forceinline__ uint32_t warp_sum(uint32_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ uint32_t warp_upto(uint32_t x) {  // inclusive prefix sum over the lanes
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
template <int T>
__device__ __forceinline__ Line make_line(const PagedAttnParams& p, bool tell) {
  const int lane = threadIdx.x & 31;
  Line l;
  l.mine = lane < p.b.B ? seq_stages<T>(p, lane, tell) : 0;
  const uint32_t upto = warp_upto(l.mine);
  l.before = upto - l.mine;
  l.total = __shfl_sync(0xffffffffu, upto, 31);
  if (p.b.B > 32) {
    uint32_t sum = 0;
#pragma unroll 1
    for (int b = 32 + lane; b < p.b.B; b += 32) sum += seq_stages<T>(p, b, tell);
    l.total += warp_sum(sum);
  }
  const uint32_t n = (uint32_t)(p.n_cta * p.quantum);
  l.per = ((l.total + n - 1) / n) * p.quantum;
  return l;
}
// The sequence that stage x < total lies in, and the stage at which its first unit begins.
template <int T>
__device__ __forceinline__ int line_find(const PagedAttnParams& p, const Line& l, uint32_t x, uint32_t& begin) {
  const int lane = threadIdx.x & 31;
  uint32_t past = __ballot_sync(0xffffffffu, l.before + l.mine > x);
  if (past) {
    const int at = __ffs(past) - 1;
    begin = __shfl_sync(0xffffffffu, l.before, at);
    return at;
  }
  uint32_t before = __shfl_sync(0xffffffffu, l.before + l.mine, 31);
#pragma unroll 1
  for (int b0 = 32; b0 < p.b.B; b0 += 32) {
    const uint32_t mine = b0 + lane < p.b.B ? seq_stages<T>(p, b0 + lane, false) : 0;
    const uint32_t upto = before + warp_upto(mine);
    past = __ballot_sync(0xffffffffu, upto > x);
    if (past) {
      const int at = __ffs(past) - 1;
      begin = __shfl_sync(0xffffffffu, upto - mine, at);
      return b0 + at;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  begin = before;
  return p.b.B - 1;
}

__device__ __forceinline__ void store_row(const PagedAttnParams& p, int64_t tok, int head, float lse2) {
  if (p.lse != nullptr) p.lse[tok * p.Hq + head] = lse2;
}

constexpr float kLn2 = 0.6931471805599453f;
// Natural logarithm of the sum whose weights are 2^(z - m + 15).
// A row without a maximum saw nothing (l = 0), or NaN logits only (l is NaN).
__device__ __forceinline__ float lse_of(float m, float l) { return m == -INFINITY ? (l == 0.f ? -INFINITY : l) : (m - 15.f + log2f(l)) * kLn2; }
// What a part with maximum pm and sum pl weighs beside the largest maximum m.
__device__ __forceinline__ float part_weight(float pm, float pl, float m) { return m == -INFINITY ? pl : exp2_fast(pm - m) * pl; }

__device__ __forceinline__ void store_joined(const PagedAttnParams& p, int64_t tok, int hd, int D, int c, const float4& y,
                                             float m, float l) {
  *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + (int64_t)hd * D + 4 * c) =
      make_uint2(pack_out(y.x, y.y, p.half), pack_out(y.z, y.w, p.half));
  if (c == 0) store_row(p, tok, hd, lse_of(m, l));
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

template <class... A>
cudaError_t launch_clusters(void (*f)(A...), dim3 grid, int cluster, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  c.attrs = attr;
  c.numAttrs = 2;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&c, f, args...);
}

}  // namespace
}  // namespace hyb
