// The gated delta rule: S := a S, S := S + k (beta (v - S^T k))^T, o = scale S^T q, a = exp(g).
#include <cuda_fp16.h>

#include "hyb_device.cuh"
#include "k_delta.h"

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

template <int DK>
struct Piece {
  uint4 w[DK / 32];  // DK / 4 bf16 in a row
  __device__ __forceinline__ void load(const uint16_t* p) {
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
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
    v = __ldg(reinterpret_cast<const uint2*>(p.v + (int64_t)t * p.v_stride + (int64_t)hv * p.DV + col));
    g = __ldg(p.g + (int64_t)t * p.Hv + hv);
    beta = __ldg(p.beta + (int64_t)t * p.Hv + hv);
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
// One CTA takes a (sequence, head).  Four warps prepare the next chunk (its rows into shared memory, K K^T and
// Q K^T, T = (I + A)^-1 by 16 x 16 inverses and block products in 32 bits) while the others take the chunk before
// through the state.  Those hold the state transposed, 16 of its columns a warp, as matrix accumulators, and work on
// the transposed equations, in which each product's result is the next one's left operand in the registers it is
// in: X^T = S^T K^T, W^T = (V^T - X^T diag(e^G)) diag(beta), U^T = W^T T^T, O^T, S^T += U^T K.
//
// Operands are f16.  Rows of K and Q are divided by powers of two kappa that put their largest element in [1, 2), so
// they go in exactly (but for elements below 2^-17 of it); S, W and T as two f16 parts, 22 bits, after S and W
// are divided by powers of two of each column of the state (sigma, omega), so that values of any size keep
// them.  Only O, whose result has 8 bits, takes single parts of S, U and P.  Sums are in 32 bits.  Errors of the
// state stay near those of 32-bit arithmetic.

constexpr int kC = 64;

template <int DK, int DV>
struct ChunkGeo {
  static constexpr int kScan = DV / 16, kPrep = 4;  // warps
  static constexpr int kThreads = (kScan + kPrep) * 32;
  // one chunk: K, Q [64][DK] f16, V [64][DV] bf16, T [64][64] in two parts, P [64][64], and seven rows of 64 factors
  static constexpr int kK = 0, kQ = kK + kC * DK * 2, kV = kQ + kC * DK * 2, kT = kV + kC * DV * 2, kP = kT + 2 * kC * kC * 2,
                       kE = kP + kC * kC * 2, kBytes = kE + 7 * kC * 4;
  static constexpr int kLd = kC + 4;  // row of A in floats
  static constexpr int kA = 2 * kBytes, kTmp = kA + kC * kLd * 4, kG = kTmp + 32 * 36 * 4, kTotal = kG + 3 * kC * 4;
};
// The factors' rows: e^G; beta e^G kappa; beta; kappa; e^(G_C - G); scale kappa of q; e^G_C
enum { kDecay, kForget, kBeta, kKappa, kLeft, kOut, kWhole };

// Byte offset of 16-byte piece c of row r in a tile with rows of `pieces` pieces: moved so that 8 rows' pieces of one
// column lie in different banks.
template <int PIECES>
__device__ __forceinline__ int tile_at(int r, int c) {
  return (r * PIECES + (c ^ (r & 7))) * 16;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

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
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_half(x, y);
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack_half(x - b.x, y - b.y);
}
// The left operand of a k-step from two accumulator tiles.
__device__ __forceinline__ void split_a(const float (&c)[4], const float (&d)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c[0], c[1], hi[0], lo[0]);
  split2(c[2], c[3], hi[1], lo[1]);
  split2(d[0], d[1], hi[2], lo[2]);
  split2(d[2], d[3], hi[3], lo[3]);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Exponent field of x, held to [lo, hi] (NaN and infinity: hi), and its power of two.
__device__ __forceinline__ uint32_t field_of(float x, uint32_t lo, uint32_t hi) { return min(max(__float_as_uint(x) >> 23, lo), hi); }
__device__ __forceinline__ float pow2_of(uint32_t e) { return __uint_as_float(e << 23); }

// Rows of K or Q: loaded, divided by their kappa and stored as f16.  16-byte pieces of a row lie in DK / 8 lanes.
template <int DK, int N>
struct RowPieces {
  uint4 w[N];
  __device__ __forceinline__ void load(const uint16_t* src, int64_t stride, int row, int n, int tid) {
    constexpr int kPieces = DK / 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = tid + 128 * i, r = at / kPieces, c = at % kPieces;
      w[i] = r < n ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)(row + r) * stride + c * 8)) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile, float* kappa, int tid) {
    constexpr int kPieces = DK / 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = tid + 128 * i, r = at / kPieces, c = at % kPieces;
      const uint32_t z[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t top = 0;  // magnitudes of bf16 order as integers
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(z[e] & 0x7fffu, (z[e] >> 16) & 0x7fffu));
#pragma unroll
      for (int o = 1; o < kPieces; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t e = min(max(top >> 7, 1u), 253u);
      const float inv = pow2_of(254u - e);
      uint32_t y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = pack_half(bf16_lo(z[x]) * inv, bf16_hi(z[x]) * inv);
      *reinterpret_cast<uint4*>(tile + tile_at<kPieces>(r, c)) = make_uint4(y[0], y[1], y[2], y[3]);
      if (c == 0) kappa[r] = pow2_of(e);
    }
  }
};

template <int DK, int DV>
__device__ __forceinline__ void chunk_prepare(const DeltaParams& p, uint8_t* smem, uint8_t* buf, int row, int n, int next, int hk, int hv, int tid) {
  using Geo = ChunkGeo<DK, DV>;
  constexpr int kLd = Geo::kLd, kPieces = DK / 8;
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t sm = smem_u32(buf);
  float* E = reinterpret_cast<float*>(buf + Geo::kE);
  float* Ghi = reinterpret_cast<float*>(smem + Geo::kG);
  float* Glo = Ghi + kC;
  float* kq = Glo + kC;
  // the chunk's rows; past its end zeros
  RowPieces<DK, DK / 16> K, Q;
  K.load(p.k + (int64_t)hk * DK, p.k_stride, row, n, tid);
  Q.load(p.q + (int64_t)hk * DK, p.q_stride, row, n, tid);
#pragma unroll
  for (int i = tid; i < kC * (DV / 8); i += 128) {
    const int r = i / (DV / 8), c = i % (DV / 8);
    const bool there = r < n;
    cp_async16(sm + Geo::kV + tile_at<DV / 8>(r, c), p.v + (int64_t)(row + (there ? r : 0)) * p.v_stride + (int64_t)hv * DV + c * 8,
               there ? 16 : 0);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // the chunk after this one on its way into L2, a line of 128 bytes at a time
  for (int i = tid; i < next * (DK / 64); i += 128) {
    const int64_t r = row + kC + i / (DK / 64);
    const int c = i % (DK / 64) * 64;
    prefetch_l2(p.k + r * p.k_stride + (int64_t)hk * DK + c);
    prefetch_l2(p.q + r * p.q_stride + (int64_t)hk * DK + c);
  }
  for (int i = tid; i < next * (DV / 64); i += 128)
    prefetch_l2(p.v + (int64_t)(row + kC + i / (DV / 64)) * p.v_stride + (int64_t)hv * DV + i % (DV / 64) * 64);
  // the sums of g in powers of two and in 64 bits, kept as two floats so that their differences keep 32; a
  // decay of e^-200 is 0 in 32 bits like any stronger one.  Two tokens a lane.
  const int r0 = 2 * lane, r1 = r0 + 1;
  float b0 = 0.f, b1 = 0.f;
  if (warp == 0) {
    const int64_t at = (int64_t)(row + r0) * p.Hv + hv;
    const float g0 = r0 < n ? p.g[at] : 0.f, g1 = r1 < n ? p.g[at + p.Hv] : 0.f;
    b0 = r0 < n ? p.beta[at] : 0.f, b1 = r1 < n ? p.beta[at + p.Hv] : 0.f;
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
    E[kDecay * kC + r0] = exp2f((float)s0), E[kDecay * kC + r1] = exp2f((float)sum);
    E[kLeft * kC + r0] = exp2f((float)(end - s0)), E[kLeft * kC + r1] = exp2f((float)(end - sum));
    E[kBeta * kC + r0] = b0, E[kBeta * kC + r1] = b1;
    if (lane == 0) E[kWhole * kC] = exp2f((float)end);
  }
  K.store(buf + Geo::kK, E + kKappa * kC, tid);
  Q.store(buf + Geo::kQ, kq, tid);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  bar_sync(5, 128);
  if (warp == 0) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = r0 + x;
      E[kForget * kC + r] = (x ? b1 : b0) * E[kDecay * kC + r] * E[kKappa * kC + r];
      E[kOut * kC + r] = p.scale * kq[r];
    }
  }

  // K K^T and Q K^T: this warp's 16 rows against the columns up to them
  float* A = reinterpret_cast<float*>(smem + Geo::kA);
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
  const int tiles = 2 * warp + 2;
#pragma unroll 2
  for (int ks = 0; ks < DK / 16; ks += 2) {
    uint32_t a[2][4], c[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int at = tile_at<kPieces>(16 * warp + (lane & 15), 2 * (ks + x) + (lane >> 4));
      ldsm_x4(sm + Geo::kK + at, a[x][0], a[x][1], a[x][2], a[x][3]);
      ldsm_x4(sm + Geo::kQ + at, c[x][0], c[x][1], c[x][2], c[x][3]);
    }
    uint32_t b[8][4];  // both k-steps
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < tiles)
        ldsm_x4(sm + Geo::kK + tile_at<kPieces>(8 * j + (lane & 7), 2 * ks + (lane >> 3)), b[j][0], b[j][1], b[j][2], b[j][3]);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < tiles) {
          mma_f16(kk[j], a[x], b[j][2 * x], b[j][2 * x + 1]);
          mma_f16(qk[j], c[x], b[j][2 * x], b[j][2 * x + 1]);
        }
  }
  const int y0 = 16 * warp + g;
  const float yh[2] = {Ghi[y0], Ghi[y0 + 8]}, yl[2] = {Glo[y0], Glo[y0 + 8]};
  const float yb[2] = {E[kBeta * kC + y0] * E[kKappa * kC + y0], E[kBeta * kC + y0 + 8] * E[kKappa * kC + y0 + 8]};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = 8 * j + 2 * t;
    const float2 xh = *reinterpret_cast<const float2*>(Ghi + x), xl = *reinterpret_cast<const float2*>(Glo + x);
    const float2 xk = *reinterpret_cast<const float2*>(E + kKappa * kC + x);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int y = y0 + 8 * r;
      float a[2] = {0.f, 0.f}, c[2] = {0.f, 0.f};
      if (j < tiles) {
        const float d0 = exp2_fast((yh[r] - xh.x) + (yl[r] - xl.x)), d1 = exp2_fast((yh[r] - xh.y) + (yl[r] - xl.y));
        a[0] = x < y ? yb[r] * xk.x * (kk[j][2 * r] * d0) : 0.f;
        a[1] = x + 1 < y ? yb[r] * xk.y * (kk[j][2 * r + 1] * d1) : 0.f;
        c[0] = x <= y ? qk[j][2 * r] * d0 : 0.f;
        c[1] = x + 1 <= y ? qk[j][2 * r + 1] * d1 : 0.f;
      }
      *reinterpret_cast<float2*>(A + y * kLd + x) = make_float2(a[0], a[1]);
      *reinterpret_cast<uint32_t*>(buf + Geo::kP + tile_at<8>(y, j) + 4 * t) = pack_half(c[0], c[1]);
    }
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
      for (int l = 0; l < i; ++l) s -= D[i * kLd + l] * x[l];
      x[i] = s;
    }
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) D[i * kLd + c] = x[i];
    }
  }
  bar_sync(5, 128);
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
    bar_sync(5, 128);
    *reinterpret_cast<float4*>(D + (16 + y) * kLd + x) = product(D + (16 + y) * kLd + 16, H, 20, -1.f);
    bar_sync(5, 128);
  }
  {
    const int y = (tid >> 3) * 2, x = (tid & 7) * 4;  // two rows and 4 columns
    auto product = [&](const float* left, const float* right, int ld, float (&s)[2][4]) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
#pragma unroll
      for (int l = 0; l < 32; l += 4) {
        const float4 u = *reinterpret_cast<const float4*>(left + l), w = *reinterpret_cast<const float4*>(left + kLd + l);
        const float a[4] = {u.x, u.y, u.z, u.w}, c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(right + (l + i) * ld + x);
          s[0][0] += a[i] * b.x, s[0][1] += a[i] * b.y, s[0][2] += a[i] * b.z, s[0][3] += a[i] * b.w;
          s[1][0] += c[i] * b.x, s[1][1] += c[i] * b.y, s[1][2] += c[i] * b.z, s[1][3] += c[i] * b.w;
        }
      }
    };
    float s[2][4];
    product(A + (32 + y) * kLd, A, kLd, s);
#pragma unroll
    for (int r = 0; r < 2; ++r) *reinterpret_cast<float4*>(M + (y + r) * 36 + x) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    bar_sync(5, 128);
    product(A + (32 + y) * kLd + 32, M, 36, s);
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float4*>(A + (32 + y + r) * kLd + x) = make_float4(-s[r][0], -s[r][1], -s[r][2], -s[r][3]);
    bar_sync(5, 128);
  }
  // T in two parts; zeros above the diagonal
#pragma unroll
  for (int i = tid; i < kC * 8; i += 128) {
    const int y = i >> 3, c = i & 7;
    const float4 u = *reinterpret_cast<const float4*>(A + y * kLd + 8 * c), w = *reinterpret_cast<const float4*>(A + y * kLd + 8 * c + 4);
    const float a[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = 8 * c + 2 * e;
      split2(x <= y ? a[2 * e] : 0.f, x + 1 <= y ? a[2 * e + 1] : 0.f, hi[e], lo[e]);
    }
    const int at = tile_at<8>(y, c);
    *reinterpret_cast<uint4*>(buf + Geo::kT + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(buf + Geo::kT + kC * kC * 2 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(ChunkGeo<DK, DV>::kThreads, 1) delta_chunks_kernel(const DeltaParams p) {
  using Geo = ChunkGeo<DK, DV>;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait_primary();
  pdl_allow_dependents();
  const int b = blockIdx.x / p.Hv, hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Run run = read_run(p, b, hv == 0 && tid == 0);
  if (run.n <= 0) return;
  const int chunks = (run.n + kC - 1) / kC;

  // barriers 1, 2: a buffer is full; 3, 4: it is free again; 5: the preparing warps' own
  if (warp >= Geo::kScan) {
    for (int c = 0; c < chunks; ++c) {
      if (c >= 2) bar_sync(3 + (c & 1), Geo::kThreads);
      chunk_prepare<DK, DV>(p, smem, smem + (c & 1) * Geo::kBytes, run.t0 + c * kC, min(run.n - c * kC, kC),
                            min(max(run.n - (c + 1) * kC, 0), kC), hk, hv, tid - Geo::kScan * 32);
      __threadfence_block();
      bar_arrive(1 + (c & 1), Geo::kThreads);
      if (c + 1 < chunks) bar_sync(5, 128);  // A is read no more
    }
    return;
  }

  // The warp's 16 columns of the state, transposed and divided by unit[]: rows (columns of S) g and g + 8, keys
  // 8 j + 2 t and the next.
  const int dv0 = 16 * warp;
  float* state = p.state + ((int64_t)run.slot * p.Hv + hv) * DK * DV + dv0;
  float S[DK / 8][4], unit[2] = {1.f, 1.f};
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[j][e] = state[(int64_t)(8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)];

  for (int c = 0; c < chunks; ++c) {
    uint8_t* buf = smem + (c & 1) * Geo::kBytes;
    const uint32_t sm = smem_u32(buf);
    const float* E = reinterpret_cast<const float*>(buf + Geo::kE) + 2 * t;  // this lane's tokens: + 8 j
    constexpr int kPieces = DK / 8;
    // sigma: the largest element of each column goes to [2^6, 2^7)
    float sig[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < DK / 8; ++j) top = fmaxf(top, fmaxf(fabsf(S[j][2 * r]), fabsf(S[j][2 * r + 1])));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      sig[r] = pow2_of(field_of(top * unit[r], 127 - 30, 127 + 110) - 6);
      const float f = unit[r] / sig[r];
#pragma unroll
      for (int j = 0; j < DK / 8; ++j) S[j][2 * r] *= f, S[j][2 * r + 1] *= f;
    }
    bar_sync(1 + (c & 1), Geo::kThreads);
    float X[8][4];  // 8 tiles of 8 tokens
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * ks], S[2 * ks + 1], hi, lo);
      uint32_t x[4][4];  // two token tiles each
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ldsm_x4(sm + Geo::kK + tile_at<kPieces>(16 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1)), x[j][0], x[j][1],
                x[j][2], x[j][3]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mma_f16(X[j], hi, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mma_f16(X[j], lo, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
    }
    // W^T = (V^T - X^T diag(e^G)) diag(beta), and its omega
    const float inv[2] = {1.f / sig[0], 1.f / sig[1]};
    float most[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t v[4];  // tokens 8 j .., columns g; columns g + 8; the next tile's
      ldsm_x4_t(sm + Geo::kV + tile_at<DV / 8>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * warp + ((lane >> 3) & 1)), v[0], v[1], v[2],
                v[3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 f = *reinterpret_cast<const float2*>(E + kForget * kC + 8 * (j + e));
        const float2 w = *reinterpret_cast<const float2*>(E + kBeta * kC + 8 * (j + e));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          X[j + e][2 * r] = bf16_lo(v[2 * e + r]) * inv[r] * w.x - X[j + e][2 * r] * f.x;
          X[j + e][2 * r + 1] = bf16_hi(v[2 * e + r]) * inv[r] * w.y - X[j + e][2 * r + 1] * f.y;
          most[r] = fmaxf(most[r], fmaxf(fabsf(X[j + e][2 * r]), fabsf(X[j + e][2 * r + 1])));
        }
      }
    }
    float om[2], back[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 1));
      most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 2));
      om[r] = pow2_of(field_of(most[r], 127 - 60, 127 + 96) - 6);
      back[r] = 1.f / om[r];
    }
    // U^T = W^T T^T: T is lower triangular, so tokens 8 j .. take k-steps up to j / 2
    float U[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[j][e] = 0.f, X[j][e] *= back[e >> 1];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t hi[4], lo[4];
      split_a(X[2 * ks], X[2 * ks + 1], hi, lo);
      auto tiles = [&](int part, const uint32_t (&a)[4], const uint32_t (&c)[4], bool both) {
        uint32_t x[4][4];
#pragma unroll
        for (int j = ks; j < 4; ++j)
          ldsm_x4(sm + part + tile_at<8>(16 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1)), x[j][0], x[j][1], x[j][2],
                  x[j][3]);
#pragma unroll
        for (int j = 2 * ks; j < 8; ++j) mma_f16(U[j], a, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
        if (!both) return;
#pragma unroll
        for (int j = 2 * ks; j < 8; ++j) mma_f16(U[j], c, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
      };
      tiles(Geo::kT, hi, lo, true);
      tiles(Geo::kT + kC * kC * 2, hi, hi, false);
    }
    // O^T = S^T Q^T diag(e^G) + U^T P^T, and S^T = e^G_C S^T + U^T diag(kappa e^(G_C - G)) K, in units of sigma omega
    float O[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      const uint32_t hi[4] = {pack_half(S[2 * ks][0], S[2 * ks][1]), pack_half(S[2 * ks][2], S[2 * ks][3]),
                              pack_half(S[2 * ks + 1][0], S[2 * ks + 1][1]), pack_half(S[2 * ks + 1][2], S[2 * ks + 1][3])};
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t x[4];
        ldsm_x4(sm + Geo::kQ + tile_at<kPieces>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1)), x[0], x[1], x[2],
                x[3]);
        mma_f16(O[j], hi, x[0], x[1]);
        mma_f16(O[j + 1], hi, x[2], x[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 d = *reinterpret_cast<const float2*>(E + kDecay * kC + 8 * j);
      const float2 k = *reinterpret_cast<const float2*>(E + kKappa * kC + 8 * j);
      O[j][0] *= d.x * back[0], O[j][1] *= d.y * back[0], O[j][2] *= d.x * back[1], O[j][3] *= d.y * back[1];
      U[j][0] *= k.x, U[j][1] *= k.y, U[j][2] *= k.x, U[j][3] *= k.y;
    }
    const float whole = E[kWhole * kC - 2 * t];
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] *= whole * back[e >> 1];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const uint32_t u[4] = {pack_half(U[2 * ks][0], U[2 * ks][1]), pack_half(U[2 * ks][2], U[2 * ks][3]),
                             pack_half(U[2 * ks + 1][0], U[2 * ks + 1][1]), pack_half(U[2 * ks + 1][2], U[2 * ks + 1][3])};
#pragma unroll
      for (int j = 2 * ks; j < 8; j += 2) {
        uint32_t x[4];
        ldsm_x4(sm + Geo::kP + tile_at<8>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1)), x[0], x[1], x[2], x[3]);
        mma_f16(O[j], u, x[0], x[1]);
        mma_f16(O[j + 1], u, x[2], x[3]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 l = *reinterpret_cast<const float2*>(E + kLeft * kC + 8 * (2 * ks + e));
        U[2 * ks + e][0] *= l.x, U[2 * ks + e][1] *= l.y, U[2 * ks + e][2] *= l.x, U[2 * ks + e][3] *= l.y;
      }
      uint32_t hi[4], lo[4];
      split_a(U[2 * ks], U[2 * ks + 1], hi, lo);
#pragma unroll
      for (int part = 0; part < DK / 8; part += 8) {
        uint32_t x[4][4];  // K as [token][key]: tokens 16 ks .., keys 8 j .. and the next 8
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ldsm_x4_t(sm + Geo::kK + tile_at<kPieces>(16 * ks + (lane & 15), part + 2 * j + (lane >> 4)), x[j][0], x[j][1], x[j][2],
                    x[j][3]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma_f16(S[part + j], hi, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma_f16(S[part + j], lo, x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
      }
    }
    unit[0] = sig[0] * om[0], unit[1] = sig[1] * om[1];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 s = *reinterpret_cast<const float2*>(E + kOut * kC + 8 * j);
      O[j][0] *= s.x * unit[0], O[j][1] *= s.y * unit[0], O[j][2] *= s.x * unit[1], O[j][3] *= s.y * unit[1];
    }
    if (c + 2 < chunks) bar_arrive(3 + (c & 1), Geo::kThreads);
    // the outputs, back in token order
    const int n = min(run.n - c * kC, kC);
    uint16_t* out = p.out + (int64_t)(run.t0 + c * kC) * p.out_stride + (int64_t)hv * DV + dv0 + 2 * t;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = transpose8(pack_bf16(O[j][0], O[j][1])), d = transpose8(pack_bf16(O[j][2], O[j][3]));
      if (8 * j + g < n) {
        uint16_t* to = out + (int64_t)(8 * j + g) * p.out_stride;
        *reinterpret_cast<uint32_t*>(to) = a;
        *reinterpret_cast<uint32_t*>(to + 8) = d;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      state[(int64_t)(8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)] = S[j][e] * unit[e >> 1];
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

template <int DK, int DV>
cudaError_t chunks(const DeltaParams& p, cudaStream_t s) {
  return launch(delta_chunks_kernel<DK, DV>, p.B * p.Hv, ChunkGeo<DK, DV>::kThreads, ChunkGeo<DK, DV>::kTotal, p, s);
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaParams& p, cudaStream_t s) {
  return launch(p.DK == 128 ? delta_steps_kernel<128> : delta_steps_kernel<64>, p.B * p.Hv, p.DV, 0, p, s);
}

cudaError_t launch_delta_chunks(const DeltaParams& p, cudaStream_t s) {
  if (p.DK == 128) return p.DV == 128 ? chunks<128, 128>(p, s) : chunks<128, 64>(p, s);
  return p.DV == 128 ? chunks<64, 128>(p, s) : chunks<64, 64>(p, s);
}

}  // namespace hyb
