// The gated delta rule: S := a S, S := S + k (beta (v - S^T k))^T, o = scale S^T q, a = exp(g).
//
// The kernels start before the one before them on the stream has ended (and wait for it before they read anything), so
// what they read may still be written while they run: plain loads only, none by the path of read-only data.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "hyb_device.cuh"
#include "k_delta.h"
#include "k_tcgen05.cuh"

namespace hyb {
namespace {

__device__ __forceinline__ void raise(uint32_t* status, uint32_t bit) {
  if (status != nullptr) atomicOr(status, bit);
}

// A sequence's rows and state, held within what the caller said; n = 0 where there is nothing to do.
struct Run {
  int t0, n, slot;
};
__device__ __forceinline__ Run read_run(const DeltaParams& p, int b, bool tell) {
  Run r;
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  r.slot = p.slots != nullptr ? p.slots[b] : b;
  r.t0 = min(max(c0, 0), p.n_new);
  const int t1 = min(max(c1, r.t0), p.n_new);
  r.n = min(t1 - r.t0, p.max_new);
  if (tell && (r.t0 != c0 || r.n != c1 - c0)) raise(p.status, HYB_STATUS_BAD_LENGTH);
  if (r.slot < 0 || r.slot >= p.n_slots) {
    if (tell && r.slot != -1) raise(p.status, HYB_STATUS_BAD_SLOT);
    r.n = 0;
  }
  return r;
}

// ---- token by token ---------------------------------------------------------------------------------
//
// Bound by the state's bytes: a warp holds 32 columns of the state in registers (each lane 4 columns of DK / 4
// rows in a run, so its keys are a contiguous piece of k), reads and writes it once, and takes the tokens
// through it.  S^T k and S^T q of the old state come from one pass over the registers:
// u = beta (v - a S^T k), o = scale (a S^T q + (k . q) u), and the second pass forms a S + k u^T.
// 64 sequences of 32 heads of 128 x 128, one token: 45 us, 6.0 TB/s; one sequence: 4.6 us, latency.  More tokens take
// 0.75 us each for one sequence, 5.5 for 32: the next token's rows are asked for behind the last use of the present ones.

template <int DK>
struct Piece {
  uint4 w[DK / 32];  // DK / 4 bf16 in a row
  __device__ __forceinline__ void load(const uint16_t* p) {
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) w[i] = *(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint4& u = w[i / 8];
    const uint32_t x = (i % 8) < 2 ? u.x : (i % 8) < 4 ? u.y : (i % 8) < 6 ? u.z : u.w;
    return i & 1 ? bf16_hi(x) : bf16_lo(x);
  }
};

template <int DK>
__global__ void __launch_bounds__(128) delta_steps_kernel(const DeltaParams p) {
  constexpr int kRows = DK / 4;  // of a lane
  pdl_wait_primary();
  pdl_allow_dependents();
  const int b = blockIdx.x / p.Hv, hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = (lane >> 3) * kRows, col = warp * 32 + (lane & 7) * 4;
  const Run r = read_run(p, b, hv == 0 && threadIdx.x == 0);
  if (r.n <= 0) return;
  float* state = p.state + (((int64_t)r.slot * p.Hv + hv) * DK + row0) * p.DV + col;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) S[i] = *reinterpret_cast<const float4*>(state + (int64_t)i * p.DV);
  Piece<DK> k, q;
  uint2 v;
  float g, beta;
  auto fetch = [&](int t) {
    k.load(p.k + (int64_t)t * p.k_stride + (int64_t)hk * DK + row0);
    q.load(p.q + (int64_t)t * p.q_stride + (int64_t)hk * DK + row0);
    v = *reinterpret_cast<const uint2*>(p.v + (int64_t)t * p.v_stride + (int64_t)hv * p.DV + col);
    g = p.g[(int64_t)t * p.Hv + hv];
    beta = p.beta[(int64_t)t * p.Hv + hv];
  };
  fetch(r.t0);
  for (int t = r.t0; t < r.t0 + r.n; ++t) {
    float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, kq = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float ki = k.at(i), qi = q.at(i);
      sk[0] += S[i].x * ki, sk[1] += S[i].y * ki, sk[2] += S[i].z * ki, sk[3] += S[i].w * ki;
      sq[0] += S[i].x * qi, sq[1] += S[i].y * qi, sq[2] += S[i].z * qi, sq[3] += S[i].w * qi;
      kq += ki * qi;
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sk[c] += __shfl_xor_sync(0xffffffffu, sk[c], o);
        sq[c] += __shfl_xor_sync(0xffffffffu, sq[c], o);
      }
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
    }
    const float a = expf(g);
    const float vf[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
    float u[4], y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u[c] = beta * (vf[c] - a * sk[c]);
      y[c] = p.scale * (a * sq[c] + kq * u[c]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float ki = k.at(i);
      S[i].x = a * S[i].x + ki * u[0];
      S[i].y = a * S[i].y + ki * u[1];
      S[i].z = a * S[i].z + ki * u[2];
      S[i].w = a * S[i].w + ki * u[3];
    }
    if (lane < 8)
      *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.out_stride + (int64_t)hv * p.DV + col) =
          make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    if (t + 1 < r.t0 + r.n) fetch(t + 1);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) *reinterpret_cast<float4*>(state + (int64_t)i * p.DV) = S[i];
}

// ---- in chunks of 64 tokens -----------------------------------------------------------------------------
//
// Within a chunk, with G_t the sum of g up to t, the updates u_t = beta_t (v_t - (state before t)^T k_t, decayed)
// satisfy (I + A) U = diag(beta) (V - diag(e^G) K S),  A_ts = beta_t e^(G_t - G_s) k_t . k_s for s < t,
// with S the state before the chunk.  Then
//   O = scale (diag(e^G) Q S + P U),  P_ts = e^(G_t - G_s) q_t . k_s for s <= t,
//   S := e^(G_C) S + K^T diag(e^(G_C - G)) U.
// One CTA takes a (sequence, head).  Two groups of four warps prepare chunks in turn, into three places of shared memory:
// the rows of K and Q, K K^T and Q K^T (on the warps' own matrix instructions, only blocks on and below the diagonal),
// T = (I + A)^-1 by 16 x 16 inverses and block products in 32 bits.  Eight warps take the chunks through the state on
// tcgen05.  They hold it transposed in tensor memory, a lane a column of the state, so that the 128 columns are the 128
// rows of every product and each product's result, read by the lanes it is in and written back as f16, is the next
// one's left operand:
//   X^T = S^T K^T,  W^T = (V^T - X^T diag(e^G)) diag(beta),  U^T = W^T T^T,
//   O^T = S^T Q^T diag(e^G) + U^T P^T,  S^T := e^(G_C) S^T + U^T diag(e^(G_C - G)) K.
// (A value dimension of 64 leaves the other 64 rows at zero.)  The outputs of a chunk are read while the next one's X is
// under way, and S decays while U is.
//
// Operands are f16.  Rows of K and Q are divided by powers of two kappa that put their largest element in [1, 2), so
// they go in exactly (but for elements below 2^-17 of it); S, W, T and the U that the state takes as two f16 parts, 22
// bits, after S and W are divided by powers of two of each column of the state (sigma, omega), so that columns keep them
// whose largest value is 2^-119 or more.  (W is formed in units of tau, sigma but at least 1, so that V divided by it
// stays finite beside a state of any smallness: 2 us of 705 below; a branch around it for states of ordinary size takes 8.)
// Only O, whose result has 8 bits, takes single parts of S, U and P.
// Sums are in 32 bits.  Errors of the state stay near those of 32-bit arithmetic.
//
// What bounds it: the chain from chunk to chunk and the instructions of both sides.  32 heads of 128 x 128 and 8192
// tokens: 700 us, 10400 clocks a chunk; the scanning warps alone 7300 (their products 1600), the preparing ones alone
// 7600, 22100 warp instructions in all.  The same products on the warps' own matrix instructions (scan of 6400 clocks at
// least) took 17800 a chunk; clusters of 4 CTAs that share the columns and pass prepared chunks on 9900 with the
// machine full, but no less where there are more than 37 heads, the copies (32 bytes a clock from an SM) being the bound.

constexpr int kC = 64, kChunkThreads = 512;  // eight scanning warps, two groups of four that prepare

template <int DK>
struct ChunkGeo {
  // one chunk: K, Q [64][DK] f16, T [64][64] in two parts, P [64][64], and seven rows of 64 factors
  static constexpr int kK = 0, kQ = kK + kC * DK * 2, kT = kQ + kC * DK * 2, kP = kT + 2 * kC * kC * 2, kE = kP + kC * kC * 2,
                       kBytes = kE + 2048;
  // three of them; each group's A, products of blocks and sums of g; columns' maxima; barriers; the tensor memory's address
  static constexpr int kLd = kC + 4;  // row of A in floats
  static constexpr int kTmp = kC * kLd * 4, kG = kTmp + 32 * 36 * 4, kWorkBytes = kG + 3 * kC * 4;
  static constexpr int kWork = 3 * kBytes, kMost = kWork + 2 * kWorkBytes, kBars = kMost + 2 * 2 * 128 * 4, kTmem = kBars + 16 * 8,
                       kTotal = kTmem + 16 + 1024;  // 1024: the tiles begin at a multiple of it
};
// Barriers: a place is full, free; products of a chunk are done
enum { kFull, kFree = 3, kDoneX = 6, kDoneU, kDoneS };
// Columns of the tensor memory: S^T; as f16, upper and lower halves; X^T, then U^T; Q S; W or U in two parts; P U
enum { kColS = 0, kColSh = 128, kColSl = 192, kColX = 256, kColQ = 320, kColW = 384, kColP = 448 };
// The factors' rows: e^G times that of q; -beta e^G kappa; beta; kappa; e^(G_C - G); scale kappa of q; e^G_C and
// the largest kappa
enum { kDecay, kForget, kBeta, kKappa, kLeft, kOut, kWhole };

// Byte offset of 16-byte piece c of row r in tiles of 64 rows of 8 pieces, moved so that 8 rows' pieces of one column lie
// in different banks (the tensor cores' 128-byte swizzle).
__device__ __forceinline__ int tile_at(int r, int c) { return (c >> 3) * 8192 + r * 128 + (((c & 7) ^ (r & 7)) * 16); }

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Two fp32 as two f16 parts.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_half(x.x, x.y);
  x = fma2(__half22float2(*reinterpret_cast<const __half2*>(&hi)), make_float2(-1.f, -1.f), x);
  lo = pack_half(x.x, x.y);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Exponent field of x, held to [lo, hi] (NaN and infinity: hi), and its power of two.
__device__ __forceinline__ uint32_t field_of(float x, uint32_t lo, uint32_t hi) { return min(max(__float_as_uint(x) >> 23, lo), hi); }
__device__ __forceinline__ float pow2_of(uint32_t e) { return __uint_as_float(e << 23); }
// 1 / x of a power of two x from 2^-126 to 2^126.
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// Rows of K or Q, four 16-byte pieces of each thread at a time: loaded, and divided by their kappa and stored as f16.
// The pieces of a row lie in DK / 8 lanes; a thread's are kRowStep rows apart, a multiple of 8, so all in one column.
template <int DK>
constexpr int kRowStep = 128 / (DK / 8);
template <int DK>
__device__ __forceinline__ void load_rows(uint4 (&w)[4], const uint16_t* src, int64_t stride, int n, int first, int tid) {
  constexpr int kPieces = DK / 8, kStep = kRowStep<DK>;
  int r = tid / kPieces + first * kStep;
  src += r * stride + tid % kPieces * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i, r += kStep, src += kStep * stride)
    w[i] = r < n ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
}
template <int DK>
__device__ __forceinline__ void store_rows(const uint4 (&w)[4], uint8_t* tile, float* kappa, int first, int tid) {
  constexpr int kPieces = DK / 8, kStep = kRowStep<DK>;
  tile += tile_at(tid / kPieces, tid % kPieces) + first * (kStep * 128);
  kappa += tid / kPieces + first * kStep;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t z[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t top = 0;  // magnitudes of bf16 order as integers
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, z[e] & 0x7fff7fffu);
#pragma unroll
    for (int o = 1; o < kPieces; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t e = min(max(max(top & 0xffffu, top >> 16) >> 7, 1u), 253u);
    const float2 inv = both(pow2_of(254u - e));
    uint32_t y[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float2 w = mul2(make_float2(bf16_lo(z[x]), bf16_hi(z[x])), inv);
      y[x] = pack_half(w.x, w.y);
    }
    *reinterpret_cast<uint4*>(tile + i * kStep * 128) = make_uint4(y[0], y[1], y[2], y[3]);
    if (tid % kPieces == 0) kappa[i * kStep] = pow2_of(e);
  }
}

// What a group has under way of its next chunk: the rows' first two steps (four pieces of each thread a step: K's, then
// Q's); the last warp two tokens' g and beta a lane.
struct Ahead {
  uint4 even[4], odd[4];
  float g0, g1, b0, b1;
};
template <int DK>
__device__ __forceinline__ void load_step(const DeltaParams& p, uint4 (&w)[4], int step, int row, int n, int hk, int tid) {
  const bool of_q = step >= DK / 64;
  const int64_t stride = of_q ? p.q_stride : p.k_stride;
  load_rows<DK>(w, (of_q ? p.q : p.k) + row * stride + (int64_t)hk * DK, stride, n, 4 * (step % (DK / 64)), tid);
}
template <int DK>
__device__ __forceinline__ void begin_chunk(const DeltaParams& p, Ahead& a, int row, int n, int hk, int hv, int tid) {
  load_step<DK>(p, a.even, 0, row, n, hk, tid);
  load_step<DK>(p, a.odd, 1, row, n, hk, tid);
  if (tid >= 96) {
    const int r0 = 2 * (tid - 96), r1 = r0 + 1;
    const int64_t at = (int64_t)(row + r0) * p.Hv + hv;
    a.g0 = r0 < n ? p.g[at] : 0.f, a.g1 = r1 < n ? p.g[at + p.Hv] : 0.f;
    a.b0 = r0 < n ? p.beta[at] : 0.f, a.b1 = r1 < n ? p.beta[at + p.Hv] : 0.f;
  }
}

// Prepares the chunk of n tokens from `row` on, which begin_chunk has begun, in `buf`; this group's next one has `next`
// tokens from row `ahead` on, and is begun here.
template <int DK>
__device__ __forceinline__ void chunk_prepare(const DeltaParams& p, uint8_t* smem, uint8_t* buf, Ahead& under_way, int barrier, int row,
                                              int n, int ahead, int next, int hk, int hv, int tid) {
  using Geo = ChunkGeo<DK>;
  constexpr int kLd = Geo::kLd;
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t sm = smem_u32(buf);
  float* E = reinterpret_cast<float*>(buf + Geo::kE);
  float* Ghi = reinterpret_cast<float*>(smem + Geo::kG);
  float* Glo = Ghi + kC;
  float* kq = Glo + kC;
  // the next chunk on its way into L2, a line of 128 bytes at a time
  for (int i = tid; i < next * (DK / 64); i += 128) {
    const int64_t r = ahead + i / (DK / 64);
    const int c = i % (DK / 64) * 64;
    prefetch_l2(p.k + r * p.k_stride + (int64_t)hk * DK + c);
    prefetch_l2(p.q + r * p.q_stride + (int64_t)hk * DK + c);
  }
  for (int i = tid; i < next * (p.DV / 64); i += 128) {
    const int lines = p.DV / 64;
    prefetch_l2(p.v + (int64_t)(ahead + i / lines) * p.v_stride + (int64_t)hv * p.DV + i % lines * 64);
  }
  // the chunk's rows, past its end zeros
#pragma unroll 1
  for (int i = 0; i < DK / 64; ++i) {
    auto store = [&](const uint4 (&w)[4], int step) {
      const bool of_q = step >= DK / 64;
      store_rows<DK>(w, buf + (of_q ? Geo::kQ : Geo::kK), of_q ? kq : E + kKappa * kC, 4 * (step % (DK / 64)), tid);
    };
    store(under_way.even, 2 * i);
    if (i + 1 < DK / 64) load_step<DK>(p, under_way.even, 2 * i + 2, row, n, hk, tid);
    store(under_way.odd, 2 * i + 1);
    if (i + 1 < DK / 64) load_step<DK>(p, under_way.odd, 2 * i + 3, row, n, hk, tid);
  }
  bar_sync(barrier, 128);
  // The sums of g in powers of two and in 64 bits, kept as two floats so that their differences keep 32; a
  // decay of e^-200 is 0 in 32 bits like any stronger one.  Two tokens a lane of the last warp, while the others begin
  // the products.
  if (warp == 3) {
    const int r0 = 2 * lane, r1 = r0 + 1;
    const float b0 = under_way.b0, b1 = under_way.b1, g0 = under_way.g0, g1 = under_way.g1;
    const double kLog2e64 = 1.4426950408889634;
    const double a = (g0 < -200.f ? -200. : (double)g0) * kLog2e64, c = (g1 < -200.f ? -200. : (double)g1) * kLog2e64;
    double sum = a + c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31), s0 = sum - c;
    Ghi[r0] = (float)s0, Ghi[r1] = (float)sum;
    Glo[r0] = (float)(s0 - (double)(float)s0), Glo[r1] = (float)(sum - (double)(float)sum);
    const float d0 = exp2f((float)s0), d1 = exp2f((float)sum), o0 = p.scale * kq[r0], o1 = p.scale * kq[r1];
    E[kForget * kC + r0] = -b0 * d0 * E[kKappa * kC + r0], E[kForget * kC + r1] = -b1 * d1 * E[kKappa * kC + r1];
    E[kOut * kC + r0] = o0, E[kOut * kC + r1] = o1;
    E[kDecay * kC + r0] = d0 * o0, E[kDecay * kC + r1] = d1 * o1;
    E[kLeft * kC + r0] = exp2f((float)(end - s0)), E[kLeft * kC + r1] = exp2f((float)(end - sum));
    E[kBeta * kC + r0] = b0, E[kBeta * kC + r1] = b1;
    if (lane == 0) E[kWhole * kC] = exp2f((float)end);
  }

  // K K^T and Q K^T below the diagonal, in blocks of 16 x 16: first this warp's own on the diagonal, then the six others in turn
  float* A = reinterpret_cast<float*>(smem);
#pragma unroll 1
  for (int i = warp; i < 10; i += 4) {
    const int bi = i < 4 ? i : i == 4 ? 1 : i < 7 ? 2 : 3, bj = i < 4 ? i : i == 4 ? 0 : i < 7 ? i - 5 : i - 7;
    float kk[2][4], qk[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t a[4], c[4], b[4];
      const int at = tile_at(16 * bi + (lane & 15), 2 * ks + (lane >> 4));
      ldsm_x4(sm + Geo::kK + at, a[0], a[1], a[2], a[3]);
      ldsm_x4(sm + Geo::kQ + at, c[0], c[1], c[2], c[3]);
      ldsm_x4(sm + Geo::kK + tile_at(16 * bj + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1)), b[0], b[1], b[2], b[3]);
      mma_f16(kk[0], a, b[0], b[1]);
      mma_f16(kk[1], a, b[2], b[3]);
      mma_f16(qk[0], c, b[0], b[1]);
      mma_f16(qk[1], c, b[2], b[3]);
    }
    if (i < 4) bar_sync(barrier, 128);  // the sums of g are there
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int y = 16 * bi + g + 8 * r;
      const float yh = Ghi[y], yl = Glo[y], yb = E[kBeta * kC + y] * E[kKappa * kC + y];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int x = 16 * bj + 8 * j + 2 * t;
        const float2 xh = *reinterpret_cast<const float2*>(Ghi + x), xl = *reinterpret_cast<const float2*>(Glo + x);
        const float2 xk = *reinterpret_cast<const float2*>(E + kKappa * kC + x);
        const float d0 = exp2_fast((yh - xh.x) + (yl - xl.x)), d1 = exp2_fast((yh - xh.y) + (yl - xl.y));
        *reinterpret_cast<float2*>(A + y * kLd + x) = make_float2(x < y ? yb * xk.x * (kk[j][2 * r] * d0) : 0.f,
                                                                  x + 1 < y ? yb * xk.y * (kk[j][2 * r + 1] * d1) : 0.f);
        *reinterpret_cast<uint32_t*>(buf + Geo::kP + tile_at(y, 2 * bj + j) + 4 * t) =
            pack_half(x <= y ? qk[j][2 * r] * d0 : 0.f, x + 1 <= y ? qk[j][2 * r + 1] * d1 : 0.f);
      }
    }
  }
  // what the products of blocks read above the diagonal
  if ((warp & 1) == 0) {
    float* z = A + (16 * warp + (lane >> 1)) * kLd + 16 * (warp + 1) + 8 * (lane & 1);
    *reinterpret_cast<float4*>(z) = *reinterpret_cast<float4*>(z + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncwarp();

  // (I + A)^-1.  Diagonal blocks of 16, one a warp, a lane a column: x_i = [i = c] - sum_l A_il x_l.
  {
    float* D = A + 16 * warp * kLd + 16 * warp;
    float x[16];
    const int c = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == c ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 d = *reinterpret_cast<const float4*>(D + i * kLd + l);
        s -= d.x * x[l];
        if (l + 1 < i) s -= d.y * x[l + 1];
        if (l + 2 < i) s -= d.z * x[l + 2];
        if (l + 3 < i) s -= d.w * x[l + 3];
      }
      x[i] = s;
    }
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) D[i * kLd + c] = x[i];
    }
  }
  bar_sync(barrier, 128);
  // Blocks of 32, then 64: the lower left of the inverse is -T22 (A21 T11).
  float* M = reinterpret_cast<float*>(smem + Geo::kTmp);
  {
    const int half = warp >> 1, me = tid & 63, y = me >> 2, x = (me & 3) * 4;  // a row and 4 columns
    float* D = A + 32 * half * kLd + 32 * half;
    float* H = M + half * 16 * 20;
    auto product = [&](const float* left, const float* right, int ld, float sign) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int l = 0; l < 16; l += 4) {
        const float4 a4 = *reinterpret_cast<const float4*>(left + l);
        const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(right + (l + i) * ld + x);
          s[0] += a[i] * b.x, s[1] += a[i] * b.y, s[2] += a[i] * b.z, s[3] += a[i] * b.w;
        }
      }
      return make_float4(sign * s[0], sign * s[1], sign * s[2], sign * s[3]);
    };
    *reinterpret_cast<float4*>(H + y * 20 + x) = product(D + (16 + y) * kLd, D, kLd, 1.f);
    bar_sync(barrier, 128);
    *reinterpret_cast<float4*>(D + (16 + y) * kLd + x) = product(D + (16 + y) * kLd + 16, H, 20, -1.f);
    bar_sync(barrier, 128);
  }
  {
    const int y = (tid >> 3) * 2, x = (tid & 7) * 4;  // two rows and 4 columns
    auto product = [&](const float* left, const float* right, int ld, float2 (&s)[2][2]) {
      s[0][0] = s[0][1] = s[1][0] = s[1][1] = both(0.f);
#pragma unroll 2
      for (int l = 0; l < 32; l += 4) {
        const float4 u = *reinterpret_cast<const float4*>(left + l), w = *reinterpret_cast<const float4*>(left + kLd + l);
        const float a[4] = {u.x, u.y, u.z, u.w}, c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(right + (l + i) * ld + x);
          const float2 b0 = make_float2(b.x, b.y), b1 = make_float2(b.z, b.w);
          s[0][0] = fma2(both(a[i]), b0, s[0][0]), s[0][1] = fma2(both(a[i]), b1, s[0][1]);
          s[1][0] = fma2(both(c[i]), b0, s[1][0]), s[1][1] = fma2(both(c[i]), b1, s[1][1]);
        }
      }
    };
    float2 s[2][2];
    product(A + (32 + y) * kLd, A, kLd, s);
#pragma unroll
    for (int r = 0; r < 2; ++r) *reinterpret_cast<float4*>(M + (y + r) * 36 + x) = make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y);
    bar_sync(barrier, 128);
    product(A + (32 + y) * kLd + 32, M, 36, s);
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float4*>(A + (32 + y + r) * kLd + x) = make_float4(-s[r][0].x, -s[r][0].y, -s[r][1].x, -s[r][1].y);
    bar_sync(barrier, 128);
  }
  if (next > 0) begin_chunk<DK>(p, under_way, ahead, next, hk, hv, tid);
  // What is done with kappa from here on takes it in units of its largest, so that what it multiplies stays near 1 for keys of
  // any size.  (The first warp has the least of what follows.)
  if (warp == 0) {
    float2* k = reinterpret_cast<float2*>(E + kKappa * kC) + lane;
    float most = fmaxf(k->x, k->y);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float inv = pow2_inverse(most);
    *k = make_float2(k->x * inv, k->y * inv);
    if (lane == 0) E[kWhole * kC + 1] = most;
  }
  // T in two parts, in blocks of 16 x 16 on and below the diagonal: two threads a row, so a warp's rows are of one block
  const int y = tid >> 1;
#pragma unroll 1
  for (int c = tid & 1; c < 2 * warp + 2; c += 2) {
    const float4 u = *reinterpret_cast<const float4*>(A + y * kLd + 8 * c), w = *reinterpret_cast<const float4*>(A + y * kLd + 8 * c + 4);
    const float a[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = 8 * c + 2 * e;
      split2(make_float2(x <= y ? a[2 * e] : 0.f, x + 1 <= y ? a[2 * e + 1] : 0.f), hi[e], lo[e]);
    }
    const int at = tile_at(y, c);
    *reinterpret_cast<uint4*>(buf + Geo::kT + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(buf + Geo::kT + kC * kC * 2 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Waits of a warp.  After one that runs out nothing waits on any; the others' run out too.
__device__ __forceinline__ bool warp_wait(const DeltaParams& p, uint64_t* bar, uint32_t parity) {
  const bool ok = __all_sync(0xffffffffu, wait_for(bar, parity));
  if (!ok && (threadIdx.x & 31) == 0) raise(p.status, HYB_STATUS_TIMEOUT);
  return ok;
}

template <int DK>
__device__ __forceinline__ void scan_chunks(const DeltaParams& p, uint8_t* smem, uint64_t* bars, uint32_t tmem, const Run& run, int hv,
                                            int chunks, int tid) {
  using Geo = ChunkGeo<DK>;
  constexpr int kKeys = DK / 2;  // of the state, a thread's; its tokens: kC / 2
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, h = warp >> 2, row = 32 * (warp & 3) + lane;
  const uint32_t sm = smem_u32(smem), mine = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  float* most_s = reinterpret_cast<float*>(smem + Geo::kMost);
  float* most_w = most_s + 256;
  const bool there = row < p.DV;
  float* state = p.state + (((int64_t)run.slot * p.Hv + hv) * DK + h * kKeys) * p.DV + row;
  // two lanes' channels of every other token: words that swap() turns into a channel's two tokens
  const int odd = lane & 1;
  const uint16_t* v0 = p.v + (int64_t)(run.t0 + 32 * h + odd) * p.v_stride + (int64_t)hv * p.DV + (row & ~1);
  uint16_t* out0 = p.out + (int64_t)(run.t0 + 32 * h + odd) * p.out_stride + (int64_t)hv * p.DV + (row & ~1);
  const uint32_t halves = odd ? 0x3276u : 0x5410u;
  auto swap = [&](uint32_t w) {  // (channel, its neighbour) of a token <-> (token, the next) of a channel
    return __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), halves);
  };
  bool alive = true, ok = true;
  float unit = 1.f, sig = 1.f, wun = 1.f;  // units of the state, of its halves, of U
  const uint32_t my_s = mine + kColS + h * kKeys;
#pragma unroll 1
  for (int i = 0; i < kKeys; i += 32) {
    uint32_t r[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = there ? __float_as_uint(state[(int64_t)(i + e) * p.DV]) : 0u;
    tmem_store32(my_s + i, r);
  }
  tmem_wait_store();

  // The outputs of chunk c: 32 tokens of this thread's channel.
  auto outputs = [&](int c) {
    const float* E = reinterpret_cast<const float*>(smem + (c % 3) * Geo::kBytes + Geo::kE) + 32 * h;
    const int n = there && alive ? run.n - c * kC - 32 * h - odd : 0;
    uint16_t* out = out0 + (int64_t)(c * kC) * p.out_stride;
    const int64_t step = 2 * p.out_stride;
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 16) {
      uint32_t q[16], u[16];
      tmem_load16(mine + kColQ + 32 * h + i0, q);
      tmem_load16(mine + kColP + 32 * h + i0, u);
      tmem_wait_load();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 d = *reinterpret_cast<const float4*>(E + kDecay * kC + i0 + i), o = *reinterpret_cast<const float4*>(E + kOut * kC + i0 + i);
        const float2 dd[2] = {make_float2(d.x, d.y), make_float2(d.z, d.w)}, oo[2] = {make_float2(o.x, o.y), make_float2(o.z, o.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = i + 2 * e;
          const float2 y = fma2(mul2(pair(q[at], q[at + 1]), both(sig)), dd[e], mul2(mul2(pair(u[at], u[at + 1]), both(wun)), oo[e]));
          u[at / 2] = pack_bf16(y.x, y.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2, out += step) {
        const uint32_t w = swap(u[i / 2]);
        if (i0 + i < n) *reinterpret_cast<uint32_t*>(out) = w;
      }
    }
    __syncwarp();
    if (lane == 0 && alive) mbar_arrive(bars + kFree + c % 3);
  };

#pragma unroll 1
  for (int c = 0;; ++c) {
    const int place = c % 3;
    if (c > 0) {
      alive = alive && warp_wait(p, bars + kDoneS, (c - 1) & 1);
      fence_after();
    }
    float s = 1.f;
    uint32_t v[16];
    const uint64_t operand = matrix_at(sm + place * Geo::kBytes, 16), across = matrix_at(sm + place * Geo::kBytes, 8192);
    if (c < chunks) {
    // sigma: the largest element of the column goes to [2^6, 2^7)
    float top = 0.f, other = 0.f;
#pragma unroll 1
    for (int i = 0; i < kKeys; i += 32) {
      uint32_t r[32];
      tmem_load(my_s + i, r);
      tmem_wait_load();
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        top = fmaxf(fmaxf(fabsf(__uint_as_float(r[e])), fabsf(__uint_as_float(r[e + 1]))), top);
        other = fmaxf(fmaxf(fabsf(__uint_as_float(r[e + 2])), fabsf(__uint_as_float(r[e + 3]))), other);
      }
    }
    top = fmaxf(top, other);
    most_s[128 * h + row] = top;
    bar_sync(2, 256);
    top = fmaxf(top, most_s[128 * (1 - h) + row]);
    s = pow2_of(field_of(top * unit, 8, 253) - 6);
    {
      const float f = fminf(unit * pow2_inverse(s), FLT_MAX);
#pragma unroll
      for (int i = 0; i < kKeys; i += 32) {
        uint32_t r[32], hi[16], lo[16];
        tmem_load(my_s + i, r);
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(mul2(pair(r[2 * e], r[2 * e + 1]), both(f)), hi[e], lo[e]);
        tmem_store16(mine + kColSh + (h * kKeys + i) / 2, hi);
        tmem_store16(mine + kColSl + (h * kKeys + i) / 2, lo);
      }
    }
    {
      const int n = there ? run.n - c * kC - 32 * h - odd : 0;
      const uint16_t* from = v0 + (int64_t)(c * kC) * p.v_stride;
      const int64_t step = 2 * p.v_stride;
#pragma unroll
      for (int i = 0; i < 16; ++i, from += step) v[i] = 2 * i < n ? *reinterpret_cast<const uint32_t*>(from) : 0u;
    }
    tmem_wait_store();
    fence_before();
    bar_sync(2, 256);
    if (warp == 0 && ok) {
      fence_after();
      ok = warp_wait(p, bars + kFull + place, (c / 3) & 1);
      if (ok && elect_one()) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)
          mma_tmem_on(tmem + kColX, tmem + kColSh + 8 * k, operand, Geo::kK + (k / 4) * 8192 + (k % 4) * 32, product_of(kC, false), k > 0);
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)
          mma_tmem_on(tmem + kColX, tmem + kColSl + 8 * k, operand, Geo::kK + (k / 4) * 8192 + (k % 4) * 32, product_of(kC, false), true);
        commit_to(bars + kDoneX);
      }
    }
    __syncwarp();
    }
    if (c > 0) outputs(c - 1);
    if (c == chunks) break;
    sig = s;
    const float* E = reinterpret_cast<const float*>(smem + place * Geo::kBytes + Geo::kE) + 32 * h;
    alive = alive && warp_wait(p, bars + kFull + place, (c / 3) & 1);
    alive = alive && warp_wait(p, bars + kDoneX, c & 1);
    fence_after();
    // W = diag(beta) (V - diag(e^G) X), and its omega
    uint32_t x[32];
    tmem_load(mine + kColX + 32 * h, x);
    tmem_wait_load();
    const float tau = fmaxf(sig, 1.f), inv = pow2_inverse(tau);
    const float2 to_tau = both(sig * inv);
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(E + kForget * kC + i), w = *reinterpret_cast<const float4*>(E + kBeta * kC + i);
      const float2 ff[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)}, ww[2] = {make_float2(w.x, w.y), make_float2(w.z, w.w)};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t two = swap(v[i / 2 + e]);
        const float2 y = fma2(mul2(pair(x[i + 2 * e], x[i + 2 * e + 1]), to_tau), ff[e], mul2(mul2(make_float2(bf16_lo(two), bf16_hi(two)), both(inv)), ww[e]));
        x[i + 2 * e] = __float_as_uint(y.x), x[i + 2 * e + 1] = __float_as_uint(y.y);
        most = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), most);
      }
    }
    most_w[128 * h + row] = most;
    bar_sync(2, 256);
    most = fmaxf(most, most_w[128 * (1 - h) + row]);
    const float om = pow2_of(field_of(most, 8, 253) - 6);
    const float back = pow2_inverse(om);
    {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) split2(mul2(pair(x[2 * i], x[2 * i + 1]), both(back)), hi[i], lo[i]);
      tmem_store16(mine + kColW + 16 * h, hi);
      tmem_store16(mine + kColW + 32 + 16 * h, lo);
    }
    tmem_wait_store();
    fence_before();
    bar_sync(2, 256);
    if (warp == 0 && ok && elect_one()) {
      fence_after();
      // U^T = W^T T^T over the place of X: tokens 16 k .. take part in those from 16 k on
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_tmem_on(tmem + kColX + 16 * k, tmem + kColW + (part == 1 ? 32 : 0) + 8 * k,
                   operand, Geo::kT + (part == 2 ? kC * kC * 2 : 0) + 2048 * k + 32 * k, product_of(kC - 16 * k, false),
                   part > 0 || k > 0);
      commit_to(bars + kDoneU);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k)
        mma_tmem_on(tmem + kColQ, tmem + kColSh + 8 * k, operand, Geo::kQ + (k / 4) * 8192 + (k % 4) * 32, product_of(kC, false), k > 0);
    }
    __syncwarp();
    // The state's new unit is the larger of its decayed part's and of U's; meanwhile it decays.
    const float whole = E[kWhole * kC - 32 * h];
    wun = tau * (om * E[kWhole * kC - 32 * h + 1]);  // U goes on times kappa
    const float now = fminf(fmaxf(fmaxf(sig * pow2_of(field_of(whole, 1, 127)), wun), pow2_of(8)), pow2_of(253));
    const float by = pow2_inverse(now);
    {
      const float f = whole * fminf(unit * by, FLT_MAX);
#pragma unroll
      for (int i = 0; i < kKeys; i += 32) {
        uint32_t r[32];
        tmem_load(my_s + i, r);
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 y = mul2(pair(r[e], r[e + 1]), both(f));
          r[e] = __float_as_uint(y.x), r[e + 1] = __float_as_uint(y.y);
        }
        tmem_store32(my_s + i, r);
      }
    }
    unit = now;
    alive = alive && warp_wait(p, bars + kDoneU, c & 1);
    fence_after();
    tmem_load(mine + kColX + 32 * h, x);
    tmem_wait_load();
    {
      const float part = wun * by;
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 k = *reinterpret_cast<const float4*>(E + kKappa * kC + i);
        const float2 y = mul2(pair(x[i], x[i + 1]), make_float2(k.x, k.y)), z = mul2(pair(x[i + 2], x[i + 3]), make_float2(k.z, k.w));
        x[i] = __float_as_uint(y.x), x[i + 1] = __float_as_uint(y.y), x[i + 2] = __float_as_uint(z.x), x[i + 3] = __float_as_uint(z.y);
        hi[i / 2] = pack_half(y.x, y.y), hi[i / 2 + 1] = pack_half(z.x, z.y);
      }
      tmem_store16(mine + kColSl + 16 * h, hi);  // its part of the outputs, in place of the state's lower halves
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 l = *reinterpret_cast<const float4*>(E + kLeft * kC + i);
        split2(mul2(pair(x[i], x[i + 1]), mul2(make_float2(l.x, l.y), both(part))), hi[i / 2], lo[i / 2]);
        split2(mul2(pair(x[i + 2], x[i + 3]), mul2(make_float2(l.z, l.w), both(part))), hi[i / 2 + 1], lo[i / 2 + 1]);
      }
      tmem_store16(mine + kColW + 16 * h, hi);
      tmem_store16(mine + kColW + 32 + 16 * h, lo);
    }
    tmem_wait_store();
    fence_before();
    bar_sync(2, 256);
    if (warp == 0 && ok && elect_one()) {
      fence_after();
      // P U, and S^T += U^T K
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_tmem_on(tmem + kColP + 16 * k, tmem + kColSl + 8 * k, operand, Geo::kP + 2048 * k + 32 * k, product_of(kC - 16 * k, false), k > 0);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_tmem_on(tmem + kColS, tmem + kColW + 32 * part + 8 * k, across, Geo::kK + 2048 * k, product_of(DK, true), true);
      commit_to(bars + kDoneS);
    }
    __syncwarp();
  }
#pragma unroll 1
  for (int i = 0; i < kKeys; i += 32) {
    uint32_t r[32];
    tmem_load(my_s + i, r);
    tmem_wait_load();
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (there && alive) state[(int64_t)(i + e) * p.DV] = __uint_as_float(r[e]) * unit;
  }
}

template <int DK>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunks_kernel(const DeltaParams p) {
  using Geo = ChunkGeo<DK>;
  extern __shared__ uint8_t raw[];
  pdl_wait_primary();
  pdl_allow_dependents();
  const int b = blockIdx.x / p.Hv, hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const int tid = threadIdx.x, warp = tid >> 5;
  const Run run = read_run(p, b, hv == 0 && tid == 0);
  if (run.n <= 0) return;
  const int chunks = (run.n + kC - 1) / kC;
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kBars);
  uint32_t* where = reinterpret_cast<uint32_t*>(smem + Geo::kTmem);
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(bars + kFull + i, 4), mbar_init(bars + kFree + i, 8);
    mbar_init(bars + kDoneX, 1);
    mbar_init(bars + kDoneU, 1);
    mbar_init(bars + kDoneS, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(where)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *where;
  if (warp < 8) {
    scan_chunks<DK>(p, smem, bars, tmem, run, hv, chunks, tid);
  } else {
    const int group = (warp - 8) >> 2, me = tid & 127;
    int* go = reinterpret_cast<int*>(smem + Geo::kTmem + 4 + 4 * group);
    Ahead under_way{};
    if (group < chunks) begin_chunk<DK>(p, under_way, run.t0 + group * kC, min(run.n - group * kC, kC), hk, hv, me);
#pragma unroll 1
    for (int c = group; c < chunks; c += 2) {
      const int place = c % 3, next = c + 2;
      if (c >= 3) {
        if (me == 0) {
          const bool ok = wait_for(bars + kFree + place, (c / 3 - 1) & 1);
          if (!ok) raise(p.status, HYB_STATUS_TIMEOUT);
          *go = ok;
        }
        bar_sync(3 + group, 128);
        if (*go == 0) break;
      }
      chunk_prepare<DK>(p, smem + Geo::kWork + group * Geo::kWorkBytes, smem + place * Geo::kBytes, under_way, 3 + group, run.t0 + c * kC,
                        min(run.n - c * kC, kC), run.t0 + next * kC, min(max(run.n - next * kC, 0), kC), hk, hv, me);
      fence_smem();
      __syncwarp();
      if ((me & 31) == 0) mbar_arrive(bars + kFull + place);
      bar_sync(3 + group, 128);  // A is read no more
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

cudaError_t launch(void (*f)(DeltaParams), int blocks, int threads, int smem, const DeltaParams& p, cudaStream_t s) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, f, p);
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaParams& p, cudaStream_t s) {
  return launch(p.DK == 128 ? delta_steps_kernel<128> : delta_steps_kernel<64>, p.B * p.Hv, p.DV, 0, p, s);
}

cudaError_t launch_delta_chunks(const DeltaParams& p, cudaStream_t s) {
  if (p.DK == 128) return launch(delta_chunks_kernel<128>, p.B * p.Hv, kChunkThreads, ChunkGeo<128>::kTotal, p, s);
  return launch(delta_chunks_kernel<64>, p.B * p.Hv, kChunkThreads, ChunkGeo<64>::kTotal, p, s);
}

}  // namespace hyb
