// The gated delta rule: S := a S, S := S + k (beta (v - S^T k))^T, o = scale S^T q, a = exp(g).
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
// Q K^T, T = (I + A)^-1 diag(beta) by 16 x 16 inverses and block products in 32 bits) while the others take the
// chunk before through the state.  Those hold the state transposed, 16 of its columns a warp, as matrix
// accumulators, and work on the transposed equations, in which each product's result is the next one's left operand
// in the registers it is in: X^T = S^T K^T, W^T = V^T - X^T diag(e^G), U^T = W^T T^T, O^T, S^T += U^T K.
// Inputs are exact in bf16; what is computed (S, W, U, T, P) goes in as two bf16 parts, 16 bits, with 32-bit
// sums, which keeps the state within about 4e-6.

constexpr int kC = 64;

template <int DK, int DV>
struct ChunkGeo {
  static constexpr int kScan = DV / 16, kPrep = 4;  // warps
  static constexpr int kThreads = (kScan + kPrep) * 32;
  // one chunk's tiles: K, Q [64][DK], V [64][DV], T and P [64][64] in two parts, all bf16; e^G scale, e^G, e^(G_C - G), e^G_C
  static constexpr int kK = 0, kQ = kK + kC * DK * 2, kV = kQ + kC * DK * 2, kT = kV + kC * DV * 2, kP = kT + 2 * kC * kC * 2,
                       kE = kP + 2 * kC * kC * 2, kBytes = kE + 4 * kC * 4;
  static constexpr int kLd = kC + 4;  // row of A in floats
  static constexpr int kA = 2 * kBytes, kTmp = kA + kC * kLd * 4, kG = kTmp + 32 * 36 * 4, kTotal = kG + kC * 8 + kC * 4;
};

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

// Two fp32 as two bf16 parts.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int DK, int DV>
__device__ void chunk_prepare(const DeltaParams& p, uint8_t* smem, uint8_t* buf, int row, int n, int hk, int hv, int tid) {
  using Geo = ChunkGeo<DK, DV>;
  constexpr int kLd = Geo::kLd;
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t sm = smem_u32(buf);
  // the chunk's rows; past its end zeros
  auto rows = [&](int off, const uint16_t* src, int64_t stride, auto pieces) {
    constexpr int kPieces = decltype(pieces)::value;
#pragma unroll
    for (int i = tid; i < kC * kPieces; i += 128) {
      const int r = i / kPieces, c = i % kPieces;
      const bool there = r < n;
      cp_async16(sm + off + tile_at<kPieces>(r, c), src + (int64_t)(row + (there ? r : 0)) * stride + c * 8, there ? 16 : 0);
    }
  };
  rows(Geo::kK, p.k + (int64_t)hk * DK, p.k_stride, std::integral_constant<int, DK / 8>());
  rows(Geo::kQ, p.q + (int64_t)hk * DK, p.q_stride, std::integral_constant<int, DK / 8>());
  rows(Geo::kV, p.v + (int64_t)hv * DV, p.v_stride, std::integral_constant<int, DV / 8>());
  asm volatile("cp.async.commit_group;" ::: "memory");

  // sums of g, in 64 bits so that their differences keep 32; a decay of e^-200 is 0 in 32 bits like any stronger one
  double* G = reinterpret_cast<double*>(smem + Geo::kG);
  float* beta = reinterpret_cast<float*>(smem + Geo::kG + kC * 8);
  float* E = reinterpret_cast<float*>(buf + Geo::kE);
  if (warp == 0) {
    const int r0 = 2 * lane, r1 = r0 + 1;
    const float g0 = r0 < n ? p.g[(int64_t)(row + r0) * p.Hv + hv] : 0.f, g1 = r1 < n ? p.g[(int64_t)(row + r1) * p.Hv + hv] : 0.f;
    const double a = g0 < -200.f ? -200. : (double)g0, c = g1 < -200.f ? -200. : (double)g1;
    double sum = a + c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    G[r0] = sum - c;
    G[r1] = sum;
    const double end = __shfl_sync(0xffffffffu, sum, 31);
    const float e0 = expf((float)(sum - c)), e1 = expf((float)sum);
    E[r0] = p.scale * e0, E[r1] = p.scale * e1;
    E[kC + r0] = e0, E[kC + r1] = e1;
    E[2 * kC + r0] = expf((float)(end - (sum - c))), E[2 * kC + r1] = expf((float)(end - sum));
    if (lane == 0) E[3 * kC] = expf((float)end);
    beta[r0] = r0 < n ? p.beta[(int64_t)(row + r0) * p.Hv + hv] : 0.f;
    beta[r1] = r1 < n ? p.beta[(int64_t)(row + r1) * p.Hv + hv] : 0.f;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  bar_sync(5, 128);

  // K K^T and Q K^T: this warp's 16 rows against the columns up to them
  float* A = reinterpret_cast<float*>(smem + Geo::kA);
  constexpr int kPieces = DK / 8;
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
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= tiles) break;
      uint32_t b[4];  // both k-steps
      ldsm_x4(sm + Geo::kK + tile_at<kPieces>(8 * j + (lane & 7), 2 * ks + (lane >> 3)), b[0], b[1], b[2], b[3]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mma_16816(kk[j], a[x][0], a[x][1], a[x][2], a[x][3], b[2 * x], b[2 * x + 1]);
        mma_16816(qk[j], c[x][0], c[x][1], c[x][2], c[x][3], b[2 * x], b[2 * x + 1]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int y = 16 * warp + g + 8 * r, x = 8 * j + 2 * t;
      float a[2] = {0.f, 0.f}, c[2] = {0.f, 0.f};
      if (j < tiles) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (x + e > y) continue;
          const float d = expf((float)(G[y] - G[x + e]));
          a[e] = x + e < y ? beta[y] * (kk[j][2 * r + e] * d) : 0.f;
          c[e] = p.scale * (qk[j][2 * r + e] * d);
        }
      }
      *reinterpret_cast<float2*>(A + y * kLd + x) = make_float2(a[0], a[1]);
      uint32_t hi, lo;
      split2(c[0], c[1], hi, lo);
      const int at = tile_at<8>(y, j) + 4 * t;
      *reinterpret_cast<uint32_t*>(buf + Geo::kP + at) = hi;
      *reinterpret_cast<uint32_t*>(buf + Geo::kP + kC * kC * 2 + at) = lo;
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
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const float a = D[(16 + y) * kLd + l];
      const float4 b = *reinterpret_cast<const float4*>(D + l * kLd + x);
      s[0] += a * b.x, s[1] += a * b.y, s[2] += a * b.z, s[3] += a * b.w;
    }
    *reinterpret_cast<float4*>(M + half * 16 * 20 + y * 20 + x) = make_float4(s[0], s[1], s[2], s[3]);
    bar_sync(5, 128);
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const float a = D[(16 + y) * kLd + 16 + l];
      const float4 b = *reinterpret_cast<const float4*>(M + half * 16 * 20 + l * 20 + x);
      s[0] -= a * b.x, s[1] -= a * b.y, s[2] -= a * b.z, s[3] -= a * b.w;
    }
    *reinterpret_cast<float4*>(D + (16 + y) * kLd + x) = make_float4(s[0], s[1], s[2], s[3]);
    bar_sync(5, 128);
  }
  {
    const int y = tid >> 2, x = (tid & 3) * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float* at, float a) {
      const float4 b = *reinterpret_cast<const float4*>(at), c = *reinterpret_cast<const float4*>(at + 4);
      s[0] += a * b.x, s[1] += a * b.y, s[2] += a * b.z, s[3] += a * b.w;
      s[4] += a * c.x, s[5] += a * c.y, s[6] += a * c.z, s[7] += a * c.w;
    };
#pragma unroll 8
    for (int l = 0; l < 32; ++l) add(A + l * kLd + x, A[(32 + y) * kLd + l]);
    float4* m = reinterpret_cast<float4*>(M + y * 36 + x);
    m[0] = make_float4(s[0], s[1], s[2], s[3]);
    m[1] = make_float4(s[4], s[5], s[6], s[7]);
    bar_sync(5, 128);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll 8
    for (int l = 0; l < 32; ++l) add(M + l * 36 + x, -A[(32 + y) * kLd + 32 + l]);
    float4* d = reinterpret_cast<float4*>(A + (32 + y) * kLd + x);
    d[0] = make_float4(s[0], s[1], s[2], s[3]);
    d[1] = make_float4(s[4], s[5], s[6], s[7]);
    bar_sync(5, 128);
  }
  // T = inverse diag(beta), in two parts; zeros above the diagonal
#pragma unroll
  for (int i = tid; i < kC * 8; i += 128) {
    const int y = i >> 3, c = i & 7;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = 8 * c + 2 * e;
      split2(x <= y ? A[y * kLd + x] * beta[x] : 0.f, x + 1 <= y ? A[y * kLd + x + 1] * beta[x + 1] : 0.f, hi[e], lo[e]);
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
  const int b = blockIdx.x / p.Hv, hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Run run = read_run(p, b, hv == 0 && tid == 0);
  if (run.n <= 0) return;
  const int chunks = (run.n + kC - 1) / kC;

  // barriers 1, 2: a buffer is full; 3, 4: it is free again; 5: the preparing warps' own
  if (warp >= Geo::kScan) {
    for (int c = 0; c < chunks; ++c) {
      if (c >= 2) bar_sync(3 + (c & 1), Geo::kThreads);
      chunk_prepare<DK, DV>(p, smem, smem + (c & 1) * Geo::kBytes, run.t0 + c * kC, min(run.n - c * kC, kC), hk, hv,
                            tid - Geo::kScan * 32);
      __threadfence_block();
      bar_arrive(1 + (c & 1), Geo::kThreads);
      if (c + 1 < chunks) bar_sync(5, 128);  // A is read no more
    }
    return;
  }

  // The warp's 16 columns of the state, transposed: rows (columns of S) g and g + 8, keys 8 j + 2 t and the next.
  const int dv0 = 16 * warp;
  float* state = p.state + ((int64_t)run.slot * p.Hv + hv) * DK * DV + dv0;
  float S[DK / 8][4];
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[j][e] = state[(int64_t)(8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)];

  for (int c = 0; c < chunks; ++c) {
    uint8_t* buf = smem + (c & 1) * Geo::kBytes;
    const uint32_t sm = smem_u32(buf);
    const float* E = reinterpret_cast<const float*>(buf + Geo::kE);
    constexpr int kPieces = DK / 8;
    bar_sync(1 + (c & 1), Geo::kThreads);
    float X[8][4], O[8][4];  // 8 tiles of 8 tokens
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[j][e] = O[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t hi[4], lo[4];
      split2(S[2 * ks][0], S[2 * ks][1], hi[0], lo[0]);
      split2(S[2 * ks][2], S[2 * ks][3], hi[1], lo[1]);
      split2(S[2 * ks + 1][0], S[2 * ks + 1][1], hi[2], lo[2]);
      split2(S[2 * ks + 1][2], S[2 * ks + 1][3], hi[3], lo[3]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t x[4], y[4];  // two token tiles
        const int at = tile_at<kPieces>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1));
        ldsm_x4(sm + Geo::kK + at, x[0], x[1], x[2], x[3]);
        ldsm_x4(sm + Geo::kQ + at, y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma_16816(X[j + e], hi[0], hi[1], hi[2], hi[3], x[2 * e], x[2 * e + 1]);
          mma_16816(X[j + e], lo[0], lo[1], lo[2], lo[3], x[2 * e], x[2 * e + 1]);
          mma_16816(O[j + e], hi[0], hi[1], hi[2], hi[3], y[2 * e], y[2 * e + 1]);
          mma_16816(O[j + e], lo[0], lo[1], lo[2], lo[3], y[2 * e], y[2 * e + 1]);
        }
      }
    }
    // W^T = V^T - X^T diag(e^G)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t v[4];  // tokens 8 j .., columns g; columns g + 8; the next tile's
      ldsm_x4_t(sm + Geo::kV + tile_at<DV / 8>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * warp + ((lane >> 3) & 1)), v[0], v[1], v[2],
                v[3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 f = *reinterpret_cast<const float2*>(E + kC + 8 * (j + e) + 2 * t);
        const float2 s = *reinterpret_cast<const float2*>(E + 8 * (j + e) + 2 * t);
        X[j + e][0] = bf16_lo(v[2 * e]) - X[j + e][0] * f.x;
        X[j + e][1] = bf16_hi(v[2 * e]) - X[j + e][1] * f.y;
        X[j + e][2] = bf16_lo(v[2 * e + 1]) - X[j + e][2] * f.x;
        X[j + e][3] = bf16_hi(v[2 * e + 1]) - X[j + e][3] * f.y;
        O[j + e][0] *= s.x, O[j + e][1] *= s.y, O[j + e][2] *= s.x, O[j + e][3] *= s.y;
      }
    }
    // U^T = W^T T^T: T is lower triangular, so tokens 8 j .. take k-steps up to j / 2
    float U[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t hi[4], lo[4];
      split2(X[2 * ks][0], X[2 * ks][1], hi[0], lo[0]);
      split2(X[2 * ks][2], X[2 * ks][3], hi[1], lo[1]);
      split2(X[2 * ks + 1][0], X[2 * ks + 1][1], hi[2], lo[2]);
      split2(X[2 * ks + 1][2], X[2 * ks + 1][3], hi[3], lo[3]);
#pragma unroll
      for (int j = 2 * ks; j < 8; j += 2) {
        uint32_t x[4], y[4];
        const int at = tile_at<8>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1));
        ldsm_x4(sm + Geo::kT + at, x[0], x[1], x[2], x[3]);
        ldsm_x4(sm + Geo::kT + kC * kC * 2 + at, y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma_16816(U[j + e], hi[0], hi[1], hi[2], hi[3], x[2 * e], x[2 * e + 1]);
          mma_16816(U[j + e], lo[0], lo[1], lo[2], lo[3], x[2 * e], x[2 * e + 1]);
          mma_16816(U[j + e], hi[0], hi[1], hi[2], hi[3], y[2 * e], y[2 * e + 1]);
        }
      }
    }
    // O^T += U^T P^T, and S^T = e^G_C S^T + U^T diag(e^(G_C - G)) K
    const float whole = E[3 * kC];
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] *= whole;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t hi[4], lo[4];
      split2(U[2 * ks][0], U[2 * ks][1], hi[0], lo[0]);
      split2(U[2 * ks][2], U[2 * ks][3], hi[1], lo[1]);
      split2(U[2 * ks + 1][0], U[2 * ks + 1][1], hi[2], lo[2]);
      split2(U[2 * ks + 1][2], U[2 * ks + 1][3], hi[3], lo[3]);
#pragma unroll
      for (int j = 2 * ks; j < 8; j += 2) {
        uint32_t x[4], y[4];
        const int at = tile_at<8>(8 * j + (lane & 7) + 8 * (lane >> 4), 2 * ks + ((lane >> 3) & 1));
        ldsm_x4(sm + Geo::kP + at, x[0], x[1], x[2], x[3]);
        ldsm_x4(sm + Geo::kP + kC * kC * 2 + at, y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma_16816(O[j + e], hi[0], hi[1], hi[2], hi[3], x[2 * e], x[2 * e + 1]);
          mma_16816(O[j + e], lo[0], lo[1], lo[2], lo[3], x[2 * e], x[2 * e + 1]);
          mma_16816(O[j + e], hi[0], hi[1], hi[2], hi[3], y[2 * e], y[2 * e + 1]);
        }
      }
      const float2 l0 = *reinterpret_cast<const float2*>(E + 2 * kC + 16 * ks + 2 * t);
      const float2 l1 = *reinterpret_cast<const float2*>(E + 2 * kC + 16 * ks + 8 + 2 * t);
      split2(U[2 * ks][0] * l0.x, U[2 * ks][1] * l0.y, hi[0], lo[0]);
      split2(U[2 * ks][2] * l0.x, U[2 * ks][3] * l0.y, hi[1], lo[1]);
      split2(U[2 * ks + 1][0] * l1.x, U[2 * ks + 1][1] * l1.y, hi[2], lo[2]);
      split2(U[2 * ks + 1][2] * l1.x, U[2 * ks + 1][3] * l1.y, hi[3], lo[3]);
#pragma unroll
      for (int j = 0; j < DK / 8; j += 2) {
        uint32_t x[4];  // K as [token][key]: tokens 16 ks .., keys 8 j .. and the next 8
        ldsm_x4_t(sm + Geo::kK + tile_at<kPieces>(16 * ks + (lane & 15), j + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma_16816(S[j + e], hi[0], hi[1], hi[2], hi[3], x[2 * e], x[2 * e + 1]);
          mma_16816(S[j + e], lo[0], lo[1], lo[2], lo[3], x[2 * e], x[2 * e + 1]);
        }
      }
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
    for (int e = 0; e < 4; ++e) state[(int64_t)(8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)] = S[j][e];
}

template <int DK, int DV>
cudaError_t chunks(const DeltaParams& p, cudaStream_t s) {
  constexpr int smem = ChunkGeo<DK, DV>::kTotal;
  const cudaError_t e = cudaFuncSetAttribute(delta_chunks_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_chunks_kernel<DK, DV><<<p.B * p.Hv, ChunkGeo<DK, DV>::kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaParams& p, cudaStream_t s) {
  if (p.DK == 128)
    delta_steps_kernel<128><<<p.B * p.Hv, p.DV, 0, s>>>(p);
  else
    delta_steps_kernel<64><<<p.B * p.Hv, p.DV, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_delta_chunks(const DeltaParams& p, cudaStream_t s) {
  if (p.DK == 128) return p.DV == 128 ? chunks<128, 128>(p, s) : chunks<128, 64>(p, s);
  return p.DV == 128 ? chunks<64, 128>(p, s) : chunks<64, 64>(p, s);
}

}  // namespace hyb
