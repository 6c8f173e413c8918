// Attention over the paged 8-bit cache for many bf16 query rows, on the tensor cores' own memory (tcgen05).
//
// A CTA takes 128 rows and passes the tokens they can see 128 at a time:
//   four converting warps turn the tile's codes into f16 in shared memory (the next tile's codes are on their way in
//     registers meanwhile);
//   four softmax warps, a thread a row, read S, keep the running maximum and sum, and write the weights P as f16
//     over the columns of S; one of their threads issues S = Q C_k^T and O += P C_v (accumulators S [128 x 128] and
//     O [128 x D] in tensor memory).
// Within a CTA the products and the softmax of a tile follow one another; two CTAs share an SM, and the one's softmax
// runs beside the other's products.  A row's maximum is followed only when a tile passes it by more than 2^8, so O is
// rescaled rarely: weights are 2^(z - m + 7) vs / ref, at most 2^15, with full 11 bits down to 2^-21 of the largest; ref is
// a row's own, from the scales of what it sees.
//
// 2047 tokens of 10001, 32 heads of 128: 580 us, 519 TFLOP/s.  Bound by the chain of a tile: the operands' way from shared
// memory and the conversions into it (about 2000 clocks a tile) beside a softmax of about 3400 when it took 606 us.  Tiles of
// 64 tokens with two accumulators of logits took 722 us when this form took 665: a product of 64 columns reads as many bytes of
// its left operand as one of 128.  Row tiles unit by unit took 665 us, all units' last ones first 639, the last turn's in parts 606.
#include "k_paged.cuh"
#include "k_tcgen05.cuh"

namespace hyb {
namespace {

constexpr int kTile = 128;  // rows, and tokens
constexpr int kGroups = kTile / 16;
constexpr int kThreads = 256;
constexpr float kGrowth = 8.f, kBase = 7.f;

template <int D>
struct MmaGeo {
  static constexpr int kQ = 0, kK = kQ + kTile * D * 2, kV = kK + kTile * D * 2, kScales = kV + kTile * D * 2;
  // two tiles' scales and live tokens of each 16-token group; barriers; the tensor memory's address
  static constexpr int kLive = kScales + 2 * 2 * kGroups * 4, kBars = kLive + 2 * kGroups * 4, kTmem = kBars + 8 * 8,
                       kTotal = kTmem + 16 + 1024;  // 1024: the tiles begin at a multiple of it
  static constexpr int kSubTile = kTile * 128;      // 64 channels of all rows
};
enum { kKFull, kKFree, kVFull, kVFree, kSFull, kOFull };

// A wait of a whole warp: one lane polls.  After a wait that runs out nothing that waits on it is done; the others'
// waits run out too, and the CTA ends.
__device__ __forceinline__ bool warp_wait(const PagedAttnParams& p, uint64_t* bar, uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    ok = wait_for(bar, parity);
    if (!ok) raise(p.status, HYB_STATUS_TIMEOUT);
  }
  __syncwarp();
  return __all_sync(0xffffffffu, ok);
}

// ---- the pieces of work of a CTA ---------------------------------------------------------------------------
// n_cta > 0: this CTA's part of the line of all units' tiles, where every sequence has at most 128 rows a KV head; as
// many pieces as units in it.  Otherwise one piece: a row tile, or a part of one of the last.  Row tiles go by what they
// see, all units' last ones first.
struct Piece {
  Seq seq;
  Span<kTile> span;
  int b, h, row0, rows, s0, s1;
  int64_t slot;   // where a part's result goes
  bool complete;  // the piece is all of its row tile's tiles
};
struct Work {
  Line line;
  uint32_t at, last, first;
  bool done;
};
__device__ __forceinline__ void start_work(const PagedAttnParams& p, Work& w) {
  w.done = false;
  if (p.n_cta > 0) {
    w.line = make_line<kTile>(p, blockIdx.x == 0 && threadIdx.x < 32);
    w.first = min(w.line.per * blockIdx.x, w.line.total);
    w.last = min(w.first + w.line.per, w.line.total);
    w.at = w.first;
  }
}
// All lanes of a warp.  False when there is no more.
__device__ __forceinline__ bool next_piece(const PagedAttnParams& p, Work& w, Piece& x) {
  bool bad;
  if (p.n_cta > 0) {
    if (w.at >= w.last) return false;
    uint32_t begin;
    x.b = line_find<kTile>(p, w.line, w.at, begin);
    x.seq = read_seq(p.b, x.b, p.c.P, &bad);
    x.span = seq_span<kTile>(p, x.seq);
    x.h = (int)((w.at - begin) / (uint32_t)x.span.stages);
    const uint32_t ubegin = begin + (uint32_t)x.h * x.span.stages;
    x.s0 = (int)(w.at - ubegin);
    x.s1 = (int)min((uint32_t)x.span.stages, w.last - ubegin);
    x.complete = x.s0 == 0 && x.s1 == x.span.stages;
    x.slot = 2 * (int64_t)blockIdx.x + (w.at == w.first ? 0 : 1);
    x.row0 = 0;
    x.rows = min(x.seq.n * p.G, kTile);
    w.at = ubegin + x.s1;
  } else {
    if (w.done) return false;
    w.done = true;
    const int units = p.b.B * p.c.Hkv, late = (int)blockIdx.x - p.n_whole;  // from 0: parts
    const int tile = late < 0 ? (int)blockIdx.x : p.n_whole + late / p.n_splits;
    const int splits = late < 0 ? 1 : p.n_splits, split = late < 0 ? 0 : late % p.n_splits;
    const int unit = tile % units;
    x.b = unit / p.c.Hkv, x.h = unit % p.c.Hkv;
    x.seq = read_seq(p.b, x.b, p.c.P, &bad);
    x.rows = x.seq.n * p.G;
    x.row0 = (p.row_tiles - 1 - tile / units) * kTile;
    if (bad && x.h == 0 && x.row0 == 0 && split == 0 && threadIdx.x == 0) raise(p.status, HYB_STATUS_BAD_LENGTH);
    if (x.row0 >= x.rows) return false;
    const int pos0 = x.seq.pos0;
    const int lo = pos0 + x.row0 / p.G, hi = pos0 + (min(x.rows, x.row0 + kTile) - 1) / p.G;
    x.span = hi >= 0 ? make_span<kTile>(max(lo, 0), hi, x.seq.cap, p.W, p.S) : Span<kTile>{0, 0, 0, 0, 0};
    x.s0 = (int)((int64_t)x.span.stages * split / splits);
    x.s1 = (int)((int64_t)x.span.stages * (split + 1) / splits);
    x.complete = splits == 1;
    x.slot = late;
  }
  return true;
}

// ---- the converting warps -----------------------------------------------------------------------------------
template <int D>
struct Pieces {
  static constexpr int kN = kTile * D / 16 / 128;  // 16-code pieces of a thread, of keys and of values
  uint4 k[kN], v[kN];
};
// The table's entry for the group of 16 tokens that begins at tok, -1 past the end.
__device__ __forceinline__ int entry_of(const PagedAttnParams& p, const int32_t* table, int tok, int end, uint32_t magic) {
  const uint32_t g = (uint32_t)tok >> 4;
  return tok < end ? table[p.c.P == 16 ? g : __umulhi(g, magic)] : -1;
}
template <bool INT8>
__device__ __forceinline__ void convert_piece(const uint4& c, uint4& lo, uint4& hi) {
  codes_f16<INT8>(c.x, lo.x, lo.y);
  codes_f16<INT8>(c.y, lo.z, lo.w);
  codes_f16<INT8>(c.z, hi.x, hi.y);
  codes_f16<INT8>(c.w, hi.z, hi.w);
}
// Stores a thread's pieces of a tile as f16: rows of 64 channels, 16-byte pieces moved by the row's number.
template <int D, bool INT8>
__device__ __forceinline__ void store_pieces(uint8_t* tile, const uint4 (&c)[Pieces<D>::kN], int tid) {
  constexpr int kPerRow = D / 16;
#pragma unroll
  for (int i = 0; i < Pieces<D>::kN; ++i) {
    const int row = tid / kPerRow + i * (128 / kPerRow), col = tid % kPerRow;
    uint4 half[2];
    convert_piece<INT8>(c[i], half[0], half[1]);
    uint8_t* at = tile + (col / 4) * MmaGeo<D>::kSubTile + row * 128;
    // the upper 64 channels' threads store their second half first, so that 8 neighbours meet 8 banks
    const int flip = D == 128 ? col / 4 : 0;
    const uint4 a = flip ? half[1] : half[0], b = flip ? half[0] : half[1];
    const int ca = 2 * (col % 4) + flip, cb = ca ^ 1;
    *reinterpret_cast<uint4*>(at + ((ca ^ (row & 7)) * 16)) = a;
    *reinterpret_cast<uint4*>(at + ((cb ^ (row & 7)) * 16)) = b;
  }
}

template <int D, bool INT8>
__device__ __forceinline__ void convert_role(const PagedAttnParams& p, uint8_t* smem, uint64_t* bars, int tid) {
  using Geo = MmaGeo<D>;
  constexpr int kN = Pieces<D>::kN, kPerRow = D / 16, kStep = 128 / kPerRow;
  const uint32_t magic = (uint32_t)(((1ull << 32) + p.c.P / 16 - 1) / (uint32_t)(p.c.P / 16));
  Work w;
  Piece x;
  start_work(p, w);
  uint32_t t = 0;  // tiles so far
#pragma unroll 1
  while (next_piece(p, w, x)) {
    if (x.s0 >= x.s1) continue;
    const int32_t* table = p.b.table + (int64_t)x.b * p.b.mp;
    Pieces<D> c;
    // the rows in which this thread's pieces of the tile to be loaded next lie (kNone: no token there), and the page of this
    // thread's group's scales
    constexpr uint32_t kNone = 0xffffffffu;
    uint32_t from[kN];
    int entry[kN], gpage = -1, base, end;
    float ks, vs;
    int live;
    auto entries = [&](int s) {
      stage_range(x.span, s, base, end);
#pragma unroll
      for (int i = 0; i < kN; ++i) entry[i] = entry_of(p, table, (base + tid / kPerRow + i * kStep) & ~15, end, magic);
      if (tid < kGroups) gpage = entry_of(p, table, base + 16 * tid, end, magic);
    };
    auto places = [&]() {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int tok = base + tid / kPerRow + i * kStep;
        const int in = tok - (p.c.P == 16 ? tok >> 4 : (int)__umulhi((uint32_t)tok >> 4, magic)) * p.c.P;
        from[i] = (uint32_t)entry[i] < (uint32_t)p.c.n_pages && tok < end
                      ? ((uint32_t)entry[i] * p.c.Hkv + x.h) * p.c.P + in
                      : kNone;
      }
      if (!INT8 && p.W > 0 && base == x.span.lo) {  // what no row sees at the window's begin: its codes may be NaN
        const Gap gap = gap_of(p, base, x.seq.pos0 + x.row0 / p.G);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int tok = base + tid / kPerRow + i * kStep;
          if (tok >= gap.gap && tok < gap.from) from[i] = kNone;
        }
      }
    };
    auto load = [&](const uint8_t* codes, uint4 (&to)[kN]) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        to[i] = from[i] != kNone ? *reinterpret_cast<const uint4*>(codes + (size_t)from[i] * D + tid % kPerRow * 16) : make_uint4(0, 0, 0, 0);
    };
    auto load_scales = [&]() {
      ks = vs = 0.f;
      live = 0;
      if (tid < kGroups && base + 16 * tid < end && (uint32_t)gpage >= (uint32_t)p.c.n_pages) {
        raise(p.status, HYB_STATUS_BAD_PAGE);
      } else if (tid < kGroups && base + 16 * tid < end) {
        ks = p.c.ks[(int64_t)gpage * p.c.Hkv + x.h];
        vs = p.c.vs[(int64_t)gpage * p.c.Hkv + x.h];
        live = min(max(end - base - 16 * tid, 0), 16);
      }
    };
    entries(x.s0);
    places();
    load(p.c.k, c.k);
    load_scales();
    load(p.c.v, c.v);
#pragma unroll 1
    for (int s = x.s0; s < x.s1; ++s, ++t) {
      const bool more = s + 1 < x.s1;
      if (more) entries(s + 1);
      if (t > 0 && !warp_wait(p, bars + kKFree, (t - 1) & 1)) return;
      store_pieces<D, INT8>(smem + Geo::kK, c.k, tid);
      if (tid < kGroups) {
        float* sc = reinterpret_cast<float*>(smem + Geo::kScales) + (t & 1) * 2 * kGroups;
        sc[tid] = ks, sc[kGroups + tid] = vs;
        reinterpret_cast<int*>(smem + Geo::kLive)[(t & 1) * kGroups + tid] = live;
      }
      fence_smem();
      mbar_arrive(bars + kKFull);
      if (more) places(), load(p.c.k, c.k), load_scales();
      if (t > 0 && !warp_wait(p, bars + kVFree, (t - 1) & 1)) return;
      store_pieces<D, INT8>(smem + Geo::kV, c.v, tid);
      fence_smem();
      mbar_arrive(bars + kVFull);
      if (more) load(p.c.v, c.v);
    }
  }
}

// ---- the products (one thread) ----------------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ bool issue_logits(uint32_t sm, uint64_t* bars, uint32_t tmem, uint32_t t) {
  using Geo = MmaGeo<D>;
  if (!wait_for(bars + kKFull, t & 1)) return false;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = (k / 4) * Geo::kSubTile + (k % 4) * 32;
    mma_smem(tmem, matrix_at(sm + Geo::kQ + off, 16), matrix_at(sm + Geo::kK + off, 16), product_of(kTile, false), k > 0);
  }
  commit_to(bars + kKFree);
  commit_to(bars + kSFull);
  mbar_arrive(bars + kSFull);  // with the products: what the converting warps wrote beside the codes
  return true;
}
template <int D>
__device__ __forceinline__ bool issue_outputs(uint32_t sm, uint64_t* bars, uint32_t tmem, uint32_t t, bool first) {
  using Geo = MmaGeo<D>;
  if (!wait_for(bars + kVFull, t & 1)) return false;
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    mma_tmem(tmem + kTile, tmem + 8 * k, matrix_at(sm + Geo::kV + k * 16 * 128, Geo::kSubTile), product_of(D, true), !first || k > 0);
  commit_to(bars + kVFree);
  return true;
}

// ---- the softmax warps -------------------------------------------------------------------------------------------
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

template <int D>
__device__ __forceinline__ void softmax_role(const PagedAttnParams& p, uint8_t* smem, uint64_t* bars, uint32_t tmem, int tid) {
  using Geo = MmaGeo<D>;
  const uint32_t sm = smem_u32(smem);
  const int warp = tid >> 5;
  const uint32_t mine = tmem + ((uint32_t)(32 * warp) << 16);  // this warp's lanes
  Work w;
  Piece x;
  start_work(p, w);
  uint32_t t = 0, pieces = 0;
  bool alive = true, ok = true;  // after a wait that ran out the warps keep the barriers' count, and wait for nothing more
#pragma unroll 1
  while (next_piece(p, w, x)) {
    const int row = x.row0 + tid, pos0 = x.seq.pos0;
    const bool there = row < x.rows, any = x.row0 + 32 * warp < x.rows;
    const int64_t tok = x.seq.t0 + (there ? row / p.G : 0);
    const int hd = x.h * p.G + (there ? row % p.G : 0);
    const int pos = there ? max(pos0 + row / p.G, -1) : -1;
    float m = -INFINITY, l = 0.f;
    uint32_t ref = 1;
    if (x.s0 < x.s1) {
      // the row's query, divided by the power of two below its largest element
      float rf;
      {
        const uint16_t* src = p.q + tok * p.q_stride + (int64_t)hd * D;
        uint4 z[D / 8];
        uint32_t most = 0;  // magnitudes of bf16 order as integers
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          z[i] = there ? *(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = __vmaxu2(most, u[e] & 0x7fff7fffu);
        }
        const uint32_t e = min(max(max(most & 0xffffu, most >> 16) >> 7, 1u), 253u);
        const float inv = pow2_of(254u - e);
        rf = pow2_of(e) * p.scale;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t u[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = pack_half(bf16_lo(u[k]) * inv, bf16_hi(u[k]) * inv);
          *reinterpret_cast<uint4*>(smem + Geo::kQ + (i / 8) * Geo::kSubTile + tid * 128 + (((i % 8) ^ (tid & 7)) * 16)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      // Q is there, and O and S of the piece before are read
      fence_smem();
      fence_before();
      rows_sync();
      if (tid == 0 && ok) {
        fence_after();
        ok = issue_logits<D>(sm, bars, tmem, t);
        if (!ok) raise(p.status, HYB_STATUS_TIMEOUT);
      }
#pragma unroll 1
      for (int s = x.s0; s < x.s1; ++s, ++t) {
        int base, end;
        stage_range(x.span, s, base, end);
        alive = alive && warp_wait(p, bars + kSFull, t & 1);
        fence_after();
        if (any && alive) {
          const float* sc = reinterpret_cast<const float*>(smem + Geo::kScales) + (t & 1) * 2 * kGroups;
          const int* live = reinterpret_cast<const int*>(smem + Geo::kLive) + (t & 1) * kGroups;
          // which of 32 tokens the row sees
          auto seen = [&](int c) {
            const int at = base + 32 * c;
            uint32_t see = low_bits(pos - at + 1) & (low_bits(live[2 * c]) | (low_bits(live[2 * c + 1]) << 16));
            if (p.W > 0) see &= ~low_bits(max(pos - at + 1, 0) - p.W) | low_bits(p.S - at);
            return see;
          };
          // The tile's maximum.  Loops are not unrolled: a warp alone on its scheduler runs straight code at the rate
          // at which it is fetched.
          float top = -INFINITY, most = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            tmem_load(mine + 32 * c, r);
            const uint32_t see = seen(c);
            const bool all = __all_sync(0xffffffffu, see == 0xffffffffu);
            float v0 = sc[kGroups + 2 * c], v1 = sc[kGroups + 2 * c + 1];
            tmem_wait_load();
            float u[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (!all) {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = (see >> i) & 1u ? r[i] : 0xff800000u;
              v0 = see & 0xffffu ? v0 : 0.f, v1 = see >> 16 ? v1 : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                u[2 * (i / 16) + e] = fmaxf(u[2 * (i / 16) + e], fmaxf(__uint_as_float(r[i + 2 * e]), __uint_as_float(r[i + 2 * e + 1])));
            // scales are not negative, so the largest product gives the largest logit
            most = fmaxf(most, fmaxf(v0, v1));
            const float u0 = fmaxf(u[0], u[1]), u1 = fmaxf(u[2], u[3]);
            top = fmaxf(top, u0 == -INFINITY ? -INFINITY : u0 * (sc[2 * c] * rf));
            top = fmaxf(top, u1 == -INFINITY ? -INFINITY : u1 * (sc[2 * c + 1] * rf));
          }
          const uint32_t now = max(ref, pow2_above(most));
          const float down = pow2_of(254u - now);
          const bool grown = m == -INFINITY ? top > m : top > m + kGrowth;
          if (__any_sync(0xffffffffu, grown || now != ref)) {
            const float mn = grown ? top : m;
            const float f = mn == m ? 1.f : exp2_fast(m - mn);  // 0 where nothing was seen before
            l *= f;
            const float o = f * (pow2_of(ref) * down);
            if (s > x.s0) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                tmem_load(mine + kTile + 32 * c, r);
                tmem_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * o);
                tmem_store32(mine + kTile + 32 * c, r);
              }
            }
            m = mn;
            ref = now;
          }
          const float shift = m == -INFINITY ? 0.f : kBase - m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32], w[16];
            tmem_load(mine + 32 * c, r);
            const uint32_t see = seen(c);
            const bool all = __all_sync(0xffffffffu, see == 0xffffffffu);
            const float f0 = sc[2 * c] * rf, f1 = sc[2 * c + 1] * rf, v0 = all || (see & 0xffffu) ? sc[kGroups + 2 * c] * down : 0.f, v1 = all || (see >> 16) ? sc[kGroups + 2 * c + 1] * down : 0.f;
            float2 add = make_float2(0.f, 0.f);
            const float2 nn = make_float2(shift, shift);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 ff = i < 16 ? make_float2(f0, f0) : make_float2(f1, f1);
              const float2 vv = i < 16 ? make_float2(v0, v0) : make_float2(v1, v1);
              float2 a = fma2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ff, nn);
              a.x = exp2_fast(a.x), a.y = exp2_fast(a.y);
              if (!all) {
                if (!((see >> i) & 1u)) a.x = 0.f;
                if (!((see >> (i + 1)) & 1u)) a.y = 0.f;
              }
              add = add2(add, a);
              const float2 b = mul2(a, vv);
              w[i / 2] = pack_half(b.x, b.y);
            }
            l += add.x + add.y;
            tmem_store16(mine + 16 * c, w);  // over columns of S that every lane of this warp has read
          }
          tmem_wait_store();
        }
        fence_before();
        rows_sync();  // all of P is there
        if (tid == 0 && ok) {
          fence_after();
          ok = issue_outputs<D>(sm, bars, tmem, t, s == x.s0);
          if (s + 1 < x.s1) {
            // S takes P's place: not before the products that read it are done
            ok = ok && wait_for(bars + kVFree, t & 1) && issue_logits<D>(sm, bars, tmem, t + 1);
          } else if (ok) {
            commit_to(bars + kOFull);
          }
          if (!ok) raise(p.status, HYB_STATUS_TIMEOUT);
        }
        __syncwarp();
      }
      alive = alive && warp_wait(p, bars + kOFull, pieces & 1);
      fence_after();
      ++pieces;
    }
    // the row's result
    const float f = l == 0.f ? 0.f : pow2_of(ref) / l;
    float* ws = p.ws + (x.slot * kTile + row - x.row0) * (D + 4);
    if (any) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        if (x.s0 < x.s1) {
          tmem_load(mine + kTile + 32 * c, r);
          tmem_wait_load();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0;
        }
        if (there && x.complete) {
          uint16_t* to = p.out + tok * p.out_stride + (int64_t)hd * D + 32 * c;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint2*>(to + i) =
                make_uint2(pack_bf16(__uint_as_float(r[i]) * f, __uint_as_float(r[i + 1]) * f),
                           pack_bf16(__uint_as_float(r[i + 2]) * f, __uint_as_float(r[i + 3]) * f));
        } else if (there) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(ws + 32 * c + i) = make_float4(__uint_as_float(r[i]) * f, __uint_as_float(r[i + 1]) * f,
                                                                      __uint_as_float(r[i + 2]) * f, __uint_as_float(r[i + 3]) * f);
        }
        __syncwarp();
      }
      // sums in the units of the other forms, whose weights begin at 2^15
      l *= 256.f;
      if (there && x.complete) store_row(p, tok, hd, lse_of(m, l));
      if (there && !x.complete) *reinterpret_cast<float2*>(ws + D) = make_float2(m, l);
    }
    fence_before();
  }
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, kMmaCtasPerSm) paged_mma_kernel(const PagedAttnParams p) {
  using Geo = MmaGeo<D>;
  extern __shared__ uint8_t raw[];
  pdl_wait_primary();
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kBars);
  uint32_t* where = reinterpret_cast<uint32_t*>(smem + Geo::kTmem);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(bars + kKFull, 128);
    mbar_init(bars + kKFree, 1);
    mbar_init(bars + kVFull, 128);
    mbar_init(bars + kVFree, 1);
    mbar_init(bars + kSFull, 2);
    mbar_init(bars + kOFull, 1);
    fence_mbar_init();
  }
  if (warp == 0) {  // S and O: 256 of the SM's 512 columns
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(where)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_allow_dependents();
  const uint32_t tmem = *where;
  if (warp < 4)
    softmax_role<D>(p, smem, bars, tmem, tid);
  else
    convert_role<D, INT8>(p, smem, bars, tid - 128);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
}

template <int D, bool INT8>
cudaError_t run(const PagedAttnParams& p, cudaStream_t s) {
  const unsigned late = (unsigned)p.b.B * p.c.Hkv * p.row_tiles - p.n_whole;
  const dim3 grid(p.n_cta > 0 ? p.n_cta : p.n_whole + late * p.n_splits);
  return launch(paged_mma_kernel<D, INT8>, grid, dim3(kThreads), MmaGeo<D>::kTotal, true, s, p);
}

}  // namespace

cudaError_t launch_paged_mma(const PagedAttnParams& p, int D, int int8, cudaStream_t s) {
  cudaError_t e;
  if (D == 128)
    e = int8 ? run<128, true>(p, s) : run<128, false>(p, s);
  else
    e = int8 ? run<64, true>(p, s) : run<64, false>(p, s);
  if (e != cudaSuccess || (p.n_cta == 0 && p.n_splits == 1)) return e;
  return p.n_cta > 0 ? launch_paged_join(p, D, kTile, s) : launch_paged_join_tiles(p, D, s);
}

}  // namespace hyb
