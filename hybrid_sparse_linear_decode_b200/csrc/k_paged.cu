// Attention over the paged 8-bit cache.
#include "k_paged.cuh"

namespace hyb {
namespace {

// With codes c and scales: k_t = ks c_t, v_t = vs c_t (ks, vs of t's page).  A
// row's logits in powers of two are z_t = (q . c_t) ks scale log2(e), its output
// sum_t 2^(z_t - m) vs c_t / sum_t 2^(z_t - m) with the running maximum m.
//
// Codes become f16 exactly.  Query rows are divided by a power of two that puts
// their largest element in [1, 2), so bf16 queries become f16 with no loss above
// 2^-17 of that element.  Weights are stored as f16(2^(z - m + 15) vs / ref) with
// ref a power of two that is at least every scale that the row has seen so far: at most
// 2^15, and full 11 bits down to 2^-29 of the largest, which is one rounding of 2^-12 a
// weight, below the output type's own.  Each row has a ref of its own: a scale of pages that
// other rows of its tile see, and it does not, has no part in it.  All sums are in 32 bits.
//
// Matrix form (mma.m16n8k16), with 8 query rows as the narrow side so that the few
// rows of a decode step fill it: S^T = C_k Q^T with 16 tokens by 8 rows, O^T = C_v^T P^T
// with 16 channels by 8 rows.  The channel order inside a k-step of the first product is
// free as long as both operands agree, and so is the order of the second product's
// output rows: a lane reads 16 bytes of a token's codes at once, each 4-byte word of a
// key is one k-step's fragment after two conversions, and the words of two
// tokens' values, their bytes interleaved, are fragments of the second product.  The
// weights get from the first product's layout to the second's by 8 x 8 transposes.

constexpr int kStageTokens = 32;
constexpr int kWarps = 4;

template <int D>
struct StageGeo {
  static constexpr int kBytes = kStageTokens * D * 2 + 32;  // K codes, V codes, scales and flags
};
// Narrow form: a team of GW warps shares the stages of a ring, each warp with 8 NT rows of its own.
template <int D, int GW>
struct NarrowGeo {
  static constexpr int kTeams = kWarps / GW;
  static constexpr int kStages = (D == 128 ? 2 : 4) * GW;
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
  g.p0 = base < end ? table[ia] : -1;
  g.p1 = base + 16 < end ? table[ib] : -1;
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

// Zeros in place of the values that no row sees at the begin of a window: their weights are 0, but their codes may be NaN.
// N threads, this one number `me`; the stage is there for all of them, and they meet afterwards.
template <int D, int N>
__device__ __forceinline__ void clear_gap(uint8_t* stage, int base, const Gap& gap, int me) {
  for (int i = me; i < (gap.from - gap.gap) * (D / 16); i += N)
    reinterpret_cast<uint4*>(stage + kStageTokens * D)[(gap.gap - base) * (D / 16) + i] = make_uint4(0, 0, 0, 0);
}

// A warp's rows: NT tiles of 8; this lane's are columns 2 t and 2 t + 1 of each (t = lane % 4).
template <int D, int NT>
struct Rows {
  float o[NT][D / 16][4];  // channels (D / 8) g + 2 j (elements 0, 1) and the next (2, 3), g = lane / 4
  float m[NT][2], l[NT][2], rf[NT][2];
  float inv[NT][2];      // 1 / the value scales' reference, a power of two
  int pos[NT][2];        // position, or -1 for a row that is not there or lies before its sequence
  int pos_min, pos_max;  // of the warp's rows that are there

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      inv[n][0] = inv[n][1] = pow2_of(253);
      l[n][0] = l[n][1] = 0.f;
    }
  }
};

// Query fragments of NT row tiles: for k-step s, channels 16 t + 4 s .. + 3 (64 more for the upper half of D = 128)
// of row g.
template <int D, int NT>
struct Queries {
  uint2 frag[NT][D / 16];
};

// The query rows' bits, under way while the first stages are found: channels 16 t .. + 15 (and 64 more) of row g.
template <int D, int NT>
struct RawRows {
  uint4 z[NT][D / 64][2];
};
template <int D, int NT>
__device__ __forceinline__ void fetch_rows(const PagedAttnParams& p, RawRows<D, NT>& raw, int t0, int h, int row_first, int rows) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = row_first + 8 * n + g;
    const bool there = row < rows;
    const int tok = there ? row / p.G : 0, head = there ? row % p.G : 0;
    const uint16_t* src = p.q + (int64_t)(t0 + tok) * p.q_stride + (int64_t)(h * p.G + head) * D + 16 * t;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        raw.z[n][hh][e] = there ? *(reinterpret_cast<const uint4*>(src + 64 * hh) + e) : make_uint4(0, 0, 0, 0);
  }
}
// Their fragments, factors and positions.
template <int D, int NT>
__device__ __forceinline__ void make_rows(const PagedAttnParams& p, const RawRows<D, NT>& raw, Queries<D, NT>& Q, Rows<D, NT>& R,
                                          int row_first, int rows, int pos0) {
  const int t = threadIdx.x & 3;
  const bool half = p.half != 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float x[D / 64][16];
    float amax = 0.f;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      const uint4 u = raw.z[n][hh][0], w = raw.z[n][hh][1];
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
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const float* y = x[s >> 2] + 4 * (s & 3);
      Q.frag[n][s] = make_uint2(pack_half(y[0] * inv, y[1] * inv), pack_half(y[2] * inv, y[3] * inv));
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      R.rf[n][c] = pow2_of(__shfl_sync(0xffffffffu, e, (2 * t + c) * 4)) * p.scale;
      const int r = row_first + 8 * n + 2 * t + c;
      R.pos[n][c] = r < rows ? max(pos0 + r / p.G, -1) : -1;
    }
  }
  R.pos_min = row_first < rows ? pos0 + row_first / p.G : 0;
  R.pos_max = row_first < rows ? pos0 + (min(rows, row_first + 8 * NT) - 1) / p.G : -1;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One stage of 32 tokens for the warp's rows.  FINE: weights as two f16 parts (22 bits), for an fp16 output,
// beside whose own rounding one of 2^-12 a weight would show.
template <int D, bool INT8, int NT, bool FINE>
__device__ __forceinline__ void do_stage(const PagedAttnParams& p, const uint8_t* stage, const Queries<D, NT>& Q,
                                         Rows<D, NT>& R, int base) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float4 sc = *reinterpret_cast<const float4*>(stage + kStageTokens * D * 2);
  const int2 live = *reinterpret_cast<const int2*>(stage + kStageTokens * D * 2 + 16);
  float s[2][NT][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
  // S^T = C_k Q^T: 16-token tile i, the lane's tokens g and g + 8, columns t and t + 4 of 16 codes
#pragma unroll
  for (int hh = 0; hh < D / 64; ++hh) {
    uint4 c[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = 8 * x + g;
      c[x] = *reinterpret_cast<const uint4*>(stage + row * D + swz<D>(row, t + 4 * hh) * 16);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = c[2 * i], w = c[2 * i + 1];
        uint32_t a[4];
        codes_f16<INT8>(k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w, a[0], a[2]);
        codes_f16<INT8>(k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w, a[1], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(s[i][n], a, Q.frag[n][hh * 4 + k].x, Q.frag[n][hh * 4 + k].y);
      }
    }
  }
  // Logits, and whether one passes its row's running maximum.  A stage that every row sees whole needs no mask.
  const bool whole = live.x == 16 && live.y == 16 && base + kStageTokens <= R.pos_min + 1 &&
                     (p.W == 0 || base > R.pos_max - p.W || base + kStageTokens <= p.S);
  float v[2][NT][2];  // value scales over the rows' references; 0 where a row sees none of the 16 tokens
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float f = (i ? sc.y : sc.x) * R.rf[n][c];
        v[i][n][c] = (i ? sc.w : sc.z) * R.inv[n][c];
        s[i][n][c] *= f;
        s[i][n][2 + c] *= f;
      }
  if (!whole) {  // a block of its own: 8 drafts of 8 sequences of up to 32768 162 us, with selects in the loop above 177
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int first = base + 16 * i, there = i ? live.y : live.x;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int pos = R.pos[n][c];
          if (there <= 0 || first > pos || (p.W > 0 && first + there - 1 <= pos - p.W && first >= p.S)) v[i][n][c] = 0.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int in = g + 8 * e, tok = first + in;
            const bool seen = in < there && tok <= pos && (p.W == 0 || tok > pos - p.W || tok < p.S);
            if (!seen) s[i][n][2 * e + c] = -INFINITY;
          }
        }
    }
  }
  float top[NT][2];
  bool moved = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      top[n][c] = fmaxf(fmaxf(s[0][n][c], s[0][n][2 + c]), fmaxf(s[1][n][c], s[1][n][2 + c]));
      moved |= top[n][c] > R.m[n][c] || fmaxf(v[0][n][c], v[1][n][c]) > 1.f;
    }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float m = top[n][c];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        m = fmaxf(R.m[n][c], m);
        f[c] = m == R.m[n][c] ? 1.f : exp2_fast(R.m[n][c] - m);  // 0 where no token was seen before
        R.m[n][c] = m;
        R.l[n][c] *= f[c];
        // a reference is at least every scale that the row sees
        const float was = R.inv[n][c];
        uint32_t ref = 254u - (__float_as_uint(was) >> 23);
        if (v[0][n][c] > 1.f) ref = max(ref, pow2_above(sc.z));
        if (v[1][n][c] > 1.f) ref = max(ref, pow2_above(sc.w));
        R.inv[n][c] = pow2_of(254u - ref);
        f[c] *= pow2_inverse(was) * R.inv[n][c];
        if (v[0][n][c] != 0.f) v[0][n][c] = sc.z * R.inv[n][c];
        if (v[1][n][c] != 0.f) v[1][n][c] = sc.w * R.inv[n][c];
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        R.o[n][j][0] *= f[0];
        R.o[n][j][1] *= f[1];
        R.o[n][j][2] *= f[0];
        R.o[n][j][3] *= f[1];
      }
    }
  }
  // Weights, rounded and transposed: b[i][n] are tokens 2 t, 2 t + 1 (and 8 more) of tile i for row g
  uint32_t b[2][NT][2], fine[FINE ? 2 : 1][FINE ? NT : 1][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // a row that has seen nothing: every logit is -inf, every weight 2^-inf
    const float m0 = R.m[n][0] == -INFINITY ? 0.f : R.m[n][0] - 15.f, m1 = R.m[n][1] == -INFINITY ? 0.f : R.m[n][1] - 15.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float w0 = exp2_fast(s[i][n][2 * e] - m0), w1 = exp2_fast(s[i][n][2 * e + 1] - m1);
        R.l[n][0] += w0;
        R.l[n][1] += w1;
        const float u0 = w0 * v[i][n][0], u1 = w1 * v[i][n][1];
        const uint32_t r = pack_half(u0, u1);
        b[i][n][e] = transpose8(r);
        if (FINE) {
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&r));
          fine[FINE ? i : 0][FINE ? n : 0][e] = transpose8(pack_half(u0 - back.x, u1 - back.y));
        }
      }
    }
  }
  // O^T += C_v^T P^T: the lane holds channels (D / 8) g .. of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of tile i
  const uint8_t* vst = stage + kStageTokens * D;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[4][D / 32];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = 16 * i + 2 * t + (x & 1) + 8 * (x >> 1);
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
        uint32_t a[4];
        codes_f16<INT8>(__byte_perm(c[0][w], c[1][w], sel), a[0], a[1]);
        codes_f16<INT8>(__byte_perm(c[2][w], c[3][w], sel), a[2], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(R.o[n][2 * w + hf], a, b[i][n][0], b[i][n][1]);
          if (FINE) mma_f16(R.o[n][2 * w + hf], a, fine[FINE ? i : 0][FINE ? n : 0][0], fine[FINE ? i : 0][FINE ? n : 0][1]);
        }
      }
  }
}

// Completes the rows' sums over the 8 lanes that share them.
template <int D, int NT>
__device__ __forceinline__ void finish_sums(Rows<D, NT>& R) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = R.l[n][c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      R.l[n][c] = l;
    }
}
// Writes column c of tile n, scaled, as the lane's D / 8 channels of a row.
template <int D, int NT>
__device__ __forceinline__ void put_row(const Rows<D, NT>& R, int n, int c, float f, float* row) {
  float* o = row + ((threadIdx.x & 31) >> 2) * (D / 8);
#pragma unroll
  for (int j = 0; j < D / 16; j += 2)
    *reinterpret_cast<float4*>(o + 2 * j) = make_float4(R.o[n][j][c] * f, R.o[n][j][2 + c] * f, R.o[n][j + 1][c] * f, R.o[n][j + 1][2 + c] * f);
}

// ---- the narrow form: up to 32 bf16 rows a KV head, 64 of fp16 ------------------------------------
//
// Bound by the codes' bytes.  The stages of all (sequence, KV head) units form one
// line that the CTAs cut into equal parts, so ragged batches keep every SM busy
// to the end; the teams of a CTA (one, two or four warps that share a ring, with 8 or
// 16 rows each) take its stages in turn and are joined at each unit's end.  A unit that
// more than one CTA worked on is joined by paged_join_kernel.  Short sequences are bound by
// latency instead: a cluster of CTAs takes each unit and joins it itself, in one launch.
//
// 8 KV heads of 128, 4 query heads each: 8 sequences of 32768 tokens 92 to 96 us from GPU to GPU, 5.6 to 5.8 TB/s (0.85 to
// 0.88 of the copies'); 4 of up to 131072, int8, 130 to 143 us, 5.1 to 5.6 TB/s; 8 draft tokens of 8 sequences of up to 32768
// 159 us, 2.3 TB/s, bound by the conversions and softmax of 32 rows; one sequence of 4096 9.4 us, latency.  Three CTAs an SM
// against two: 110 against 123 us; tiles of 8 rows instead of 16 for up to 8: 93 against 107 (8 sequences of 32768).

constexpr int kMaxCluster = kPagedMaxCluster;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared memory `at` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t in_rank(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 load_rank2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_rank4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

template <int GW>
__device__ __forceinline__ void team_sync() {
  if (GW == 1) {
    __syncwarp();
  } else if (GW == kWarps) {
    __syncthreads();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)(threadIdx.x >> 5) / GW), "n"(GW * 32) : "memory");
  }
}

template <int D, bool INT8, int NT, int GW, bool FINE>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) paged_narrow_kernel(const PagedAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTeams = NarrowGeo<D, GW>::kTeams, kRing = NarrowGeo<D, GW>::kStages, kBytes = StageGeo<D>::kBytes;
  constexpr int kRows = 8 * NT * GW;
  // a joined row's place: D floats and 4 more, so that rows begin in different banks
  constexpr int kRowFloats = D + 4;
  pdl_wait_primary();
  pdl_allow_dependents();  // they wait for this grid's end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int team = warp / GW, member = warp % GW, me = threadIdx.x % (GW * 32);
  uint8_t* ring = smem + team * kRing * kBytes;
  const uint32_t magic = (uint32_t)(((1ull << 32) + p.c.P / 16 - 1) / (uint32_t)(p.c.P / 16));

  // A cluster (p.cluster CTAs) takes one unit, its CTAs equal parts of it; otherwise CTAs take parts of the line.
  Line line{};
  uint32_t first = 0, last = 1, at = 0;
  if (p.cluster == 0) {
    line = make_line<kStageTokens>(p, blockIdx.x == 0 && threadIdx.x < 32);
    first = at = min(line.per * blockIdx.x, line.total);
    last = min(first + line.per, line.total);
  }
  while (at < last) {
    int b, h, s0, s1, slot = 0;
    bool bad, complete;
    Seq seq;
    Span<kStageTokens> span;
    if (p.cluster == 0) {
      // the unit that stage `at` lies in, and the part of it that is this CTA's
      uint32_t begin;
      b = line_find<kStageTokens>(p, line, at, begin);
      seq = read_seq(p.b, b, p.c.P, &bad);
      span = seq_span<kStageTokens>(p, seq);
      h = (int)((at - begin) / (uint32_t)span.stages);
      const uint32_t ubegin = begin + (uint32_t)h * span.stages;
      s0 = (int)(at - ubegin), s1 = (int)min((uint32_t)span.stages, last - ubegin);
      complete = s0 == 0 && s1 == span.stages;
      slot = 2 * blockIdx.x + (at == first ? 0 : 1);
      at = ubegin + s1;
    } else {
      const int unit = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
      b = unit / p.c.Hkv, h = unit % p.c.Hkv;
      seq = read_seq(p.b, b, p.c.P, &bad);
      span = seq_span<kStageTokens>(p, seq);
      const int part = (span.stages + p.cluster - 1) / p.cluster;
      s0 = min(part * rank, span.stages), s1 = min(s0 + part, span.stages);
      complete = p.cluster == 1;
      at = last;
      if (bad && h == 0 && rank == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
    }
    const int rows = min(seq.n * p.G, kRows), pos0 = seq.pos0;
    const int32_t* table = p.b.table + (int64_t)b * p.b.mp;

    // the queries, then the first stages
    RawRows<D, NT> raw;
    fetch_rows<D, NT>(p, raw, seq.t0, h, 8 * NT * member, rows);
    const int mine = s1 - s0 > team ? (s1 - s0 - team + kTeams - 1) / kTeams : 0;
    StagePages nxt;
    int base, end;
    auto find = [&](int i) {
      stage_range(span, s0 + team + i * kTeams, base, end);
      nxt = stage_pages(p, table, base, end, magic);
    };
    if (mine > 0) find(0);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
      if (i < mine) {
        issue_stage<D, GW * 32>(p, ring + i * kBytes, nxt, h, base, end, me);
        if (i + 1 < mine) find(i + 1);
      }
      cp_commit();
    }
    Rows<D, NT> R;
    Queries<D, NT> Q;
    R.clear();
    make_rows<D, NT>(p, raw, Q, R, 8 * NT * member, rows, pos0);

    int slot_in = kRing - 1, slot_out = 0;
    for (int i = 0; i < mine; ++i) {
      cp_wait<kRing - 2>();
      team_sync<GW>();  // the stage is there, and the team is done with the one before
      if (i + kRing - 1 < mine) {
        issue_stage<D, GW * 32>(p, ring + slot_in * kBytes, nxt, h, base, end, me);
        if (i + kRing < mine) find(i + kRing);
      }
      cp_commit();
      int sb, se;
      stage_range(span, s0 + team + i * kTeams, sb, se);
      if (!INT8 && p.W > 0 && sb == span.lo) {
        clear_gap<D, GW * 32>(ring + slot_out * kBytes, sb, gap_of(p, sb, pos0), me);
        team_sync<GW>();
      }
      if (sb <= R.pos_max) do_stage<D, INT8, NT, FINE>(p, ring + slot_out * kBytes, Q, R, sb);
      slot_in = slot_in + 1 == kRing ? 0 : slot_in + 1;
      slot_out = slot_out + 1 == kRing ? 0 : slot_out + 1;
    }
    cp_wait<0>();
    finish_sums<D, NT>(R);

    // Join the teams through the rings' memory: [team][row][D outputs, m, l, ref].
    __syncthreads();
    float* body = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* e = body + (team * kRows + 8 * (NT * member + n) + 2 * t + c) * kRowFloats;
        put_row<D, NT>(R, n, c, 1.f, e);
        if (g == 0) e[D] = R.m[n][c], e[D + 1] = R.l[n][c], e[D + 2] = pow2_inverse(R.inv[n][c]);
      }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
      const int row = x / (D / 4), c = x % (D / 4) * 4;
      const float* e = body + row * kRowFloats;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kTeams; ++w) m = fmaxf(m, e[w * kRows * kRowFloats + D]);
      float l = 0.f, f[kTeams];
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        f[w] = m == -INFINITY ? 0.f : exp2_fast(e[w * kRows * kRowFloats + D] - m);
        l += e[w * kRows * kRowFloats + D + 1] * f[w];
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(e + w * kRows * kRowFloats + c);
        const float k = f[w] * inv * e[w * kRows * kRowFloats + D + 2];
        y.x += o.x * k, y.y += o.y * k, y.z += o.z * k, y.w += o.w * k;
      }
      if (complete) {
        store_joined(p, seq.t0 + row / p.G, h * p.G + row % p.G, D, c / 4, y, m, l);
      } else {
        float* to = p.cluster > 0 ? body + (kTeams * kRows + row) * kRowFloats : p.ws + ((int64_t)slot * kRows + row) * (D + 4);
        *reinterpret_cast<float4*>(to + c) = y;
        if (c == 0) *reinterpret_cast<float2*>(to + D) = make_float2(m, l);
      }
    }
    __syncthreads();
    if (p.cluster > 1) {
      // Join the cluster's parts: its CTAs take the row's pieces in turn, and read each other's shared memory.
      cluster_sync();
      const int rank = blockIdx.x % p.cluster;
      const uint32_t parts = smem_u32(body + kTeams * kRows * kRowFloats);
      for (int x = rank * kWarps * 32 + threadIdx.x; x < rows * (D / 4); x += p.cluster * kWarps * 32) {
        const int row = x / (D / 4), c = x % (D / 4) * 4;
        float4 o[kMaxCluster];
        float2 e[kMaxCluster];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          e[i] = make_float2(-INFINITY, 0.f);
          o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < p.cluster) {
            const uint32_t from = in_rank(parts + row * kRowFloats * 4, i);
            e[i] = load_rank2(from + D * 4);
            o[i] = load_rank4(from + c * 4);
          }
          m = fmaxf(m, e[i].x);
        }
        float l = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          const float w = part_weight(e[i].x, e[i].y, m);
          l += w;
          y.x += w * o[i].x, y.y += w * o[i].y, y.z += w * o[i].z, y.w += w * o[i].w;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
        store_joined(p, seq.t0 + row / p.G, h * p.G + row % p.G, D, c / 4, y, m, l);
      }
      cluster_sync();  // no CTA ends while another reads its memory
    }
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
  float2 e[kJoinMost / kJoinThreads];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kJoinMost / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    e[k] = i < n ? *reinterpret_cast<const float2*>(part(i) + D) : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, e[k].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinMost / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    const float w = part_weight(e[k].x, e[k].y, m);
    if (i < n) weight[i] = w;
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

// Joins the parts of units that more than one CTA worked on, and writes the rows
// of units with no visible token.  One CTA a (unit, row).
template <int D, int T>
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
  const int stages = seq_span<T>(p, seq).stages;
  if (stages == 0) {
    pdl_wait_primary();
    if (threadIdx.x < D / 4) store_joined(p, tok, hd, D, threadIdx.x, make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
    return;
  }
  // the line up to this sequence
  const Line line = make_line<T>(p, false);
  uint32_t begin = __shfl_sync(0xffffffffu, line.before, b & 31);
  if (b >= 32) {
    uint32_t sum = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) sum += seq_stages<T>(p, i, false);
    begin = warp_sum(sum);
  }
  begin += (uint32_t)h * stages;
  const uint32_t c0 = begin / line.per, c1 = (begin + stages - 1) / line.per;
  pdl_wait_primary();
  if (c0 == c1) return;  // complete in one CTA
  const uint32_t late = c0 * line.per < begin ? 1 : 0;  // the first part is not its CTA's first
  auto part = [&](int i) -> const float* {
    return p.ws + ((int64_t)(2 * (c0 + i) + (i == 0 ? late : 0)) * tile_rows + row) * (D + 4);
  };
  const int n = (int)(c1 - c0) + 1;
  float m, l;
  const float4 y = join_parts<D>(n, part, m, l);
  if (threadIdx.x < D / 4) store_joined(p, tok, hd, D, threadIdx.x, y, m, l);
}

// Joins the parts of the row tiles from n_whole on (at most 64 parts).  One warp a row.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_tiles_kernel(const PagedAttnParams p) {
  const int units = p.b.B * p.c.Hkv, tile = p.n_whole + blockIdx.x, unit = tile % units;
  const int b = unit / p.c.Hkv, h = unit % p.c.Hkv, lane = threadIdx.x & 31, n = p.n_splits;
  const int in_tile = 4 * blockIdx.y + (threadIdx.x >> 5), row = (p.row_tiles - 1 - tile / units) * kMmaRows + in_tile;
  bool bad;
  const Seq seq = read_seq(p.b, b, p.c.P, &bad);
  pdl_wait_primary();
  if (row >= seq.n * p.G) return;
  const float* parts = p.ws + ((int64_t)blockIdx.x * n * kMmaRows + in_tile) * (D + 4);
  constexpr int64_t kNext = (int64_t)kMmaRows * (D + 4);
  float2 e[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    e[k] = lane + 32 * k < n ? *reinterpret_cast<const float2*>(parts + (lane + 32 * k) * kNext + D) : make_float2(-INFINITY, 0.f);
  float m = fmaxf(e[0].x, e[1].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float w[2], l;
#pragma unroll
  for (int k = 0; k < 2; ++k) w[k] = part_weight(e[k].x, e[k].y, m);
  l = w[0] + w[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float f = __shfl_sync(0xffffffffu, i < 32 ? w[0] : w[1], i & 31);
    if (lane < D / 4) {
      const float4 o = *reinterpret_cast<const float4*>(parts + i * kNext + 4 * lane);
      y.x += f * o.x, y.y += f * o.y, y.z += f * o.z, y.w += f * o.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
  if (lane < D / 4) store_joined(p, seq.t0 + row / p.G, h * p.G + row % p.G, D, lane, y, m, l);
}

// ---- the wide form: many fp16 rows a KV head ---------------------------------------------------------
//
// A CTA takes 64 rows, 16 a warp, and passes the stages its rows can see through
// one shared ring; every warp converts the codes itself (the conversions run
// beside the other warps' products).  Few row tiles over a long cache are cut
// into n_splits parts of their stages, joined by paged_join_rows_kernel.
// Bound by the conversions and the warps' matrix instructions: 32 heads of 128, 128 tokens of 8192 134 us, 127 TFLOP/s of
// the attention's own products (half as much again is done for the weights' second part); 2047 of 10001 1855 us, 162 TFLOP/s.

constexpr int kWideRing = 4;

template <int D, bool INT8>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) paged_wide_kernel(const PagedAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int NT = 2, kBytes = StageGeo<D>::kBytes, kRowFloats = D + 4;
  pdl_wait_primary();
  pdl_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t magic = (uint32_t)(((1ull << 32) + p.c.P / 16 - 1) / (uint32_t)(p.c.P / 16));
  const int unit = blockIdx.y, b = unit / p.c.Hkv, h = unit % p.c.Hkv;
  // the tiles that see most come first
  const int tile = (int)(gridDim.x / p.n_splits) - 1 - (int)(blockIdx.x / p.n_splits);
  const int split = blockIdx.x % p.n_splits;
  bool bad;
  const Seq seq = read_seq(p.b, b, p.c.P, &bad);
  if (bad && h == 0 && tile == 0 && split == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
  const int rows = seq.n * p.G, row0 = tile * kWideRows, pos0 = seq.pos0;
  if (row0 >= rows) return;
  const int pos_min = pos0 + row0 / p.G, pos_max = pos0 + (min(rows, row0 + kWideRows) - 1) / p.G;
  const Span<kStageTokens> span = pos_max >= 0 ? make_span<kStageTokens>(max(pos_min, 0), pos_max, seq.cap, p.W, p.S) : Span<kStageTokens>{0, 0, 0, 0, 0};
  const int s0 = (int)((int64_t)span.stages * split / p.n_splits);
  const int s1 = (int)((int64_t)span.stages * (split + 1) / p.n_splits);
  const int32_t* table = p.b.table + (int64_t)b * p.b.mp;

  RawRows<D, NT> raw;
  fetch_rows<D, NT>(p, raw, seq.t0, h, row0 + 8 * NT * warp, rows);
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
  Rows<D, NT> R;
  Queries<D, NT> Q;
  R.clear();
  make_rows<D, NT>(p, raw, Q, R, row0 + 8 * NT * warp, rows, pos0);
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
    if (!INT8 && p.W > 0 && sb == span.lo) {
      clear_gap<D, kWarps * 32>(smem + (i - s0) % kWideRing * kBytes, sb, gap_of(p, sb, pos_min), threadIdx.x);
      __syncthreads();
    }
    if (sb <= R.pos_max) do_stage<D, INT8, NT, true>(p, smem + (i - s0) % kWideRing * kBytes, Q, R, sb);
  }
  cp_wait<0>();
  finish_sums<D, NT>(R);
  // Rows leave through shared memory, 8 of a warp's at a time, so that they are stored in their own order.
  __syncthreads();
  float* body = reinterpret_cast<float*>(smem) + warp * 8 * kRowFloats;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float* e = body + (2 * t + c) * kRowFloats;
      put_row<D, NT>(R, n, c, R.l[n][c] == 0.f ? 0.f : pow2_inverse(R.inv[n][c]) / R.l[n][c], e);
      if (g == 0) e[D] = R.m[n][c], e[D + 1] = R.l[n][c];
    }
    __syncwarp();
    const int first = row0 + 8 * (NT * warp + n);
    for (int x = lane; x < 8 * (D / 4); x += 32) {
      const int rr = x / (D / 4), c = x % (D / 4) * 4, row = first + rr;
      if (row >= rows) break;
      const float* e = body + rr * kRowFloats;
      const float4 y = *reinterpret_cast<const float4*>(e + c);
      const int64_t tok = seq.t0 + row / p.G;
      const int hd = h * p.G + row % p.G;
      if (p.n_splits == 1) {
        store_joined(p, tok, hd, D, c / 4, y, e[D], e[D + 1]);
      } else {
        float* ws = p.ws + (((int64_t)split * p.b.n_new + tok) * p.Hq + hd) * (D + 4);
        *reinterpret_cast<float4*>(ws + c) = y;
        if (c == 0) *reinterpret_cast<float2*>(ws + D) = make_float2(e[D], e[D + 1]);
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

template <int D, bool INT8, int NT, int GW, bool FINE>
cudaError_t narrow(const PagedAttnParams& p, cudaStream_t s) {
  constexpr int kRows = 8 * NT * GW;
  constexpr size_t rings = (size_t)NarrowGeo<D, GW>::kTeams * NarrowGeo<D, GW>::kStages * StageGeo<D>::kBytes;
  constexpr size_t rows = (size_t)(NarrowGeo<D, GW>::kTeams + 1) * kRows * (D + 4) * sizeof(float);
  constexpr size_t smem = rings > rows ? rings : rows;
  static_assert(smem <= 74 * 1024, "three CTAs share an SM");
  const auto kernel = paged_narrow_kernel<D, INT8, NT, GW, FINE>;
  if (p.cluster > 0) return launch_clusters(kernel, dim3(p.b.B * p.c.Hkv * p.cluster), p.cluster, dim3(kWarps * 32), smem, s, p);
  cudaError_t e = launch(kernel, dim3(p.n_cta), dim3(kWarps * 32), smem, true, s, p);
  if (e != cudaSuccess) return e;
  const int n = p.b.max_new * p.G < kRows ? p.b.max_new * p.G : kRows;
  return launch(paged_join_kernel<D, kStageTokens>, dim3(p.b.B * p.c.Hkv, n), dim3(kJoinThreads), 0, true, s, p, kRows);
}
template <int D, bool INT8, bool FINE>
cudaError_t narrow(const PagedAttnParams& p, int rows, cudaStream_t s) {
  if (rows == 8) return narrow<D, INT8, 1, 1, FINE>(p, s);
  if (rows == 16) return narrow<D, INT8, 2, 1, FINE>(p, s);
  if constexpr (FINE) {
    if (rows == 64) return narrow<D, INT8, 2, 4, FINE>(p, s);
  }
  return narrow<D, INT8, 2, 2, FINE>(p, s);
}

template <int D, bool INT8>
cudaError_t wide(const PagedAttnParams& p, cudaStream_t s) {
  constexpr size_t smem = (size_t)kWideRing * StageGeo<D>::kBytes;
  static_assert(smem >= (size_t)kWarps * 8 * (D + 4) * sizeof(float), "the rows that leave fit");
  const int64_t tiles = ((int64_t)p.b.max_new * p.G + kWideRows - 1) / kWideRows;
  cudaError_t e = launch(paged_wide_kernel<D, INT8>, dim3((unsigned)(tiles * p.n_splits), p.b.B * p.c.Hkv),
                         dim3(kWarps * 32), smem, true, s, p);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  return launch(paged_join_rows_kernel<D>, dim3(p.Hq, p.b.max_new, p.b.B), dim3(kJoinThreads), 0, true, s, p);
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams& p, int D, int rows, cudaStream_t s) {
  const int n = p.b.max_new * p.G < rows ? p.b.max_new * p.G : rows;
  const dim3 grid(p.b.B * p.c.Hkv, n), block(kJoinThreads);
  if (D == 128) return launch(paged_join_kernel<128, 128>, grid, block, 0, true, s, p, rows);
  return launch(paged_join_kernel<64, 128>, grid, block, 0, true, s, p, rows);
}
cudaError_t launch_paged_join_tiles(const PagedAttnParams& p, int D, cudaStream_t s) {
  const dim3 grid(p.b.B * p.c.Hkv * p.row_tiles - p.n_whole, kMmaRows / 4), block(kJoinThreads);
  return D == 128 ? launch(paged_join_tiles_kernel<128>, grid, block, 0, true, s, p) : launch(paged_join_tiles_kernel<64>, grid, block, 0, true, s, p);
}

cudaError_t launch_paged_narrow(const PagedAttnParams& p, int D, int int8, int rows, cudaStream_t s) {
  if (p.half) {
    if (D == 128) return int8 ? narrow<128, true, true>(p, rows, s) : narrow<128, false, true>(p, rows, s);
    return int8 ? narrow<64, true, true>(p, rows, s) : narrow<64, false, true>(p, rows, s);
  }
  if (D == 128) return int8 ? narrow<128, true, false>(p, rows, s) : narrow<128, false, false>(p, rows, s);
  return int8 ? narrow<64, true, false>(p, rows, s) : narrow<64, false, false>(p, rows, s);
}

cudaError_t launch_paged_wide(const PagedAttnParams& p, int D, int int8, cudaStream_t s) {
  if (D == 128) return int8 ? wide<128, true>(p, s) : wide<128, false>(p, s);
  return int8 ? wide<64, true>(p, s) : wide<64, false>(p, s);
}

}  // namespace hyb
