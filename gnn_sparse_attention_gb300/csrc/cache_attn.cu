// cache_attn.cu -- softmax attention of single tokens over a cache in 4 or 8 bits.
//
// With K = m + s u (m, s per row and head) the scores are
//     q . k = s (q . u) + m sum(q),
// and the output is sum p (m + s u) = sum (p s) u + sum p m: levels enter the
// tensor cores as they are, and what depends on a row stays outside.  A level's
// bits, masked in place, ARE a whole number in fp16's denormal range (u 2^-24, or
// u 2^-20 for the upper nibble of a byte), which the tensor cores multiply
// exactly, so unpacking costs one logical instruction for two levels and no
// conversion.  The scale of the upper nibbles is taken out of q (scores) or of
// the finished row (output); both are powers of two.
//
// Products.  The cache is read once and each element meets G queries, so the
// kernel is bound by HBM as long as unpacking keeps up; operands come straight
// from registers (mma.sync m16n8k16: 16 rows of the cache by 8 query heads).
// Through tcgen05 every level would have to be stored to shared memory as 16
// bits first, 2 to 4 times the bytes that arrive, for products that fill a
// tenth of the legacy pipe.  S^T = K Q^T has rows of the cache as rows; P^T is
// turned by movmatrix into the right operand of O^T = V^T P^T.  A lane's elements
// of K and V are whole words of a row, since any order of the head's elements
// will do for K as long as q has the same, and for V it only names output rows.
//
// Precision.  q enters in fp16 after scaling each head by a power of two: exact
// for bf16, as a sum of two (two columns) for fp32.  p s enters in fp16 (11 bits,
// or as two for fp32), scaled by a power of two per column that follows its
// maximum.  Softmax statistics, m's terms and all sums are fp32.
//
// Split.  A warp takes tiles of 16 rows, its own running maximum and sum (moved
// only when a score exceeds it by 2^8, so a tile needs a vote and no shuffles);
// warps of a CTA, CTAs of a cluster (through distributed shared memory) and, where
// a few tokens read long caches, clusters (through the workspace) are joined.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "cache.cuh"

namespace gattn {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kTile = 16;       // rows of the cache per step of a warp
constexpr int kCols = 8;        // columns of a product: query heads (fp32: halves of four)
constexpr int kMaxCluster = 8;
constexpr float kNone = -1e30f; // running maximum before any score
// Largest p s of a column in fp16: to [kYTop, 2 kYTop) when the factor is set, so that what is
// 2^-20 of it keeps its 11 bits; set again beyond kYMax.
constexpr float kYTop = 64.f, kYMax = 32768.f;

struct AttnParams {
  CacheParams c;
  const void* Q;
  const int32_t* idx;
  void* out;
  float* lse;
  float* part;   // [units * Hkv * groups][splits][cols][D + 2]
  int groups;    // column groups of a key head
  int splits;    // clusters that share a unit
  int max_keys;
};

template <int BITS, int D>
struct Lay {
  static constexpr int RB = D * BITS / 8;   // bytes of a row
  static constexpr int KW = RB / 16;        // words of a K row that a lane holds
  static constexpr int KL = KW < 4 ? KW : 4;  // ... in one load
  static constexpr int VB = RB / 8;         // bytes of a V row that a lane holds
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int MT = D / 16;         // 16-row tiles of the output
  static constexpr int QR = D / 8;          // registers of q per lane
};

__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^(127 - exponent) as a factor: x * pow2_below(x) is in [1, 2)
__device__ __forceinline__ float pow2_below(float x) {
  const int e = (__float_as_uint(x) >> 23) & 255;
  return __uint_as_float(uint32_t(254 - clampi(e, 30, 224)) << 23);
}

// rows of a tile as a lane holds them
template <int BITS, int D>
struct Tile {
  using L = Lay<BITS, D>;
  uint32_t k[2][L::KW];  // rows kr(g), kr(g) + 8
  uint32_t v[4][L::VW];  // rows t, 4 + t, 8 + t, 12 + t
  uint2 par[2];          // of the rows of k
};

// Row of the tile that stands in product row r (r < 8; r + 8 likewise): product
// rows 2t, 2t + 1 are rows t, 4 + t, so that a warp's load of V covers four whole rows.
__device__ __forceinline__ int tile_row(int r) { return (r >> 1) + 4 * (r & 1); }

template <int BITS, int D>
__device__ __forceinline__ void load_tile(Tile<BITS, D>& x, const uint8_t* __restrict__ k,
                                          const uint8_t* __restrict__ v,
                                          const uint2* __restrict__ par, int pos, int last) {
  using L = Lay<BITS, D>;
  const int lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = min(pos + tile_row(gq) + 8 * h, last);
    const uint8_t* a = k + r * L::RB + t * (L::KL * 4);
#pragma unroll
    for (int c = 0; c < L::KW / L::KL; ++c) {
      if constexpr (L::KL == 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(a + c * 64);
        x.k[h][4 * c] = q.x; x.k[h][4 * c + 1] = q.y;
        x.k[h][4 * c + 2] = q.z; x.k[h][4 * c + 3] = q.w;
      } else if constexpr (L::KL == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(a);
        x.k[h][0] = q.x; x.k[h][1] = q.y;
      } else {
        x.k[h][0] = *reinterpret_cast<const uint32_t*>(a);
      }
    }
    x.par[h] = par[r];
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int64_t r = min(pos + 4 * h + t, last);
    const uint8_t* a = v + r * L::RB + gq * L::VB;
    if constexpr (L::VB == 16) {
      const uint4 q = *reinterpret_cast<const uint4*>(a);
      x.v[h][0] = q.x; x.v[h][1] = q.y; x.v[h][2] = q.z; x.v[h][3] = q.w;
    } else if constexpr (L::VB == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(a);
      x.v[h][0] = q.x; x.v[h][1] = q.y;
    } else if constexpr (L::VB == 4) {
      x.v[h][0] = *reinterpret_cast<const uint32_t*>(a);
    } else {
      x.v[h][0] = *reinterpret_cast<const uint16_t*>(a);
    }
  }
}

// first element of word w of a lane's K row
template <int BITS, int D>
__device__ __forceinline__ int k_elem(int w, int t) {
  using L = Lay<BITS, D>;
  return ((w / L::KL) * 64 + t * (L::KL * 4) + (w % L::KL) * 4) * 8 / BITS;
}

__device__ __forceinline__ float to_f32(const float* x) { return *x; }
__device__ __forceinline__ float to_f32(const __nv_bfloat16* x) { return __bfloat162float(*x); }

// What a warp carries along: per column (a lane's two) the reference, sums, and factors
struct Cols {
  float ref[2], l[2], m[2], vf[2];
};

template <class T, int BITS, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) cache_attn_kernel(const AttnParams p) {
  using L = Lay<BITS, D>;
  constexpr bool kSplit = sizeof(T) == 4;           // fp32: a head is two columns
  constexpr int HC = kSplit ? kCols / 2 : kCols;    // heads of a column group
  __shared__ int ids[kBlkMaxTopk];
  __shared__ int n_ids;
  __shared__ float so[kWarps][HC][D + 4];           // warps' sums; then, in [0], the CTA's
  __shared__ float sref[kWarps][HC], sl[kWarps][HC];
  __shared__ float cref[HC], cl[HC];
  const BlockGeom& g = p.c.g;
  cg::cluster_group cluster = cg::this_cluster();
  const int csize = int(cluster.num_blocks()), crank = int(cluster.block_rank());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
  const int64_t cid = blockIdx.x / csize;  // cluster
  const int split = int(cid % p.splits);
  const int64_t item = cid / p.splits;     // (unit, key head, column group)
  const int cgrp = int(item % p.groups);
  const int kh = int(item / p.groups % g.Hkv);
  const int u = int(item / p.groups / g.Hkv);
  const Unit un = unit_at(g, u);
  // every CTA of a cluster has the same unit, so all leave together
  if (un.n == 0) return;
  const Span sp = span_k(g, un.s);
  const int limit = min(g.causal ? clampi(un.pos + 1, 0, sp.len) : sp.len, p.max_keys);
  int keys = limit;
  if (p.idx) {
    if (warp == 0) {
      const int nb = (sp.len + g.block - 1) / g.block;
      const int n = block_list(p.idx + int64_t(u) * g.is_u + int64_t(kh) * g.is_h, g.topk, nb, ids);
      if (lane == 0) n_ids = list_keys(ids, n, g.block, limit);
    }
    __syncthreads();
    keys = n_ids;
  }
  const int tiles = (keys + kTile - 1) / kTile;
  const int lb = 31 - __clz(g.block);
  const int64_t row0 = int64_t(kh) * g.Nk + sp.beg;
  const uint8_t* kb = p.c.k + row0 * L::RB;
  const uint8_t* vb = p.c.v + row0 * L::RB;
  const uint2* pb = p.c.par + row0;
  const auto tile_pos = [&](int i) {
    const int at = i * kTile;
    return p.idx ? (ids[at >> lb] << lb) + (at & (g.block - 1)) : at;
  };

  // q of this lane's column, scaled to fp16's range, in the order of the words of a K row
  const int head0 = kh * g.G + cgrp * HC;
  const int heads = min(HC, g.G - cgrp * HC);
  uint32_t qf[L::QR];
  float qmul[2], qsum[2];  // of the lane's columns of a product: 2t, 2t + 1
  {
    const int hc = kSplit ? gq >> 1 : gq;
    const bool on = hc < heads;
    const T* q = static_cast<const T*>(p.Q) + (int64_t(un.row) * g.H + head0 + (on ? hc : 0)) * D;
    constexpr int PW = 32 / BITS;  // elements of a word
    float f[L::KW * PW];
    float top = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < L::KW; ++w)
#pragma unroll
      for (int i = 0; i < PW; ++i) {
        const float x = on ? to_f32(q + k_elem<BITS, D>(w, t) + i) : 0.f;
        f[w * PW + i] = x;
        top = fmaxf(top, fabsf(x));
        sum += x;
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const float up = pow2_below(top) * 8192.f;  // largest element to [2^13, 2^14)
#pragma unroll
    for (int w = 0; w < L::KW; ++w)
#pragma unroll
      for (int i = 0; i < PW; i += 4) {
        // 4 bits, by the masked halves of the word: (0, 4) and (1, 5), then (2, 6) and (3, 7);
        // 8 bits: (0, 2) and (1, 3).  Upper nibbles count 16 times.
        float x[4];
        if constexpr (BITS == 4) {
          x[0] = f[w * PW + i / 2]; x[1] = f[w * PW + 4 + i / 2];
          x[2] = f[w * PW + i / 2 + 1] * 0.0625f; x[3] = f[w * PW + 4 + i / 2 + 1] * 0.0625f;
        } else {
          x[0] = f[w * PW]; x[1] = f[w * PW + 2]; x[2] = f[w * PW + 1]; x[3] = f[w * PW + 3];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] *= up;
          if (kSplit && (gq & 1)) x[e] -= __half2float(__float2half_rn(x[e]));
        }
        const int r = (w * PW + i) / 2;
        qf[r] = half2_bits(x[0], x[1]);
        qf[r + 1] = half2_bits(x[2], x[3]);
      }
    // columns 2t, 2t + 1 of a product belong to the lanes with gq = 2t, 2t + 1
    const float mul = g.qmul * 16777216.f / up, qs = sum * g.qmul;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      qmul[c] = __shfl_sync(0xffffffffu, mul, (2 * t + c) * 4);
      qsum[c] = __shfl_sync(0xffffffffu, qs, (2 * t + c) * 4);
    }
  }

  float acc[L::MT][4];
#pragma unroll
  for (int i = 0; i < L::MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  Cols cs;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    cs.ref[c] = kNone;
    cs.l[c] = cs.m[c] = 0.f;
    cs.vf[c] = 1.f;
  }

  const int nwarps = p.splits * csize * kWarps;
  const int me = (split * csize + crank) * kWarps + warp;
  constexpr int NC = kSplit ? 1 : 2;  // softmax columns of a lane
  Tile<BITS, D> cur, nxt;
  int pos = 0;
  if (me < tiles) {
    pos = tile_pos(me);
    load_tile<BITS, D>(cur, kb, vb, pb, pos, limit - 1);
  }
  for (int i = me; i < tiles; i += nwarps) {
    int npos = 0;
    if (i + nwarps < tiles) {
      npos = tile_pos(i + nwarps);
      load_tile<BITS, D>(nxt, kb, vb, pb, npos, limit - 1);
    }
    // scores
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < L::KW; ++w) {
      const uint32_t a = cur.k[0][w], b = cur.k[1][w];
      if constexpr (BITS == 4) {
        mma16816(s4, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u,
                 qf[4 * w], qf[4 * w + 1]);
        const uint32_t c = a >> 8, d = b >> 8;
        mma16816(s4, c & 0x000f000fu, d & 0x000f000fu, c & 0x00f000f0u, d & 0x00f000f0u,
                 qf[4 * w + 2], qf[4 * w + 3]);
      } else {
        mma16816(s4, a & 0x00ff00ffu, b & 0x00ff00ffu, (a >> 8) & 0x00ff00ffu,
                 (b >> 8) & 0x00ff00ffu, qf[2 * w], qf[2 * w + 1]);
      }
    }
    float lg[2][NC], sv[2], mv[2];
    bool over = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mk = __uint_as_float(cur.par[h].x << 16);
      const float sk = __uint_as_float(cur.par[h].x & 0xffff0000u);
      mv[h] = __uint_as_float(cur.par[h].y << 16);
      sv[h] = __uint_as_float(cur.par[h].y & 0xffff0000u);
      const bool in = pos + tile_row(gq) + 8 * h < limit;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float dot = kSplit ? s4[2 * h] + s4[2 * h + 1] : s4[2 * h + c];
        const float x = fmaf(dot * qmul[c], sk, mk * qsum[c]);
        lg[h][c] = in ? x : neg_inf();
        over = over || lg[h][c] > cs.ref[c] + 8.f;
      }
    }
    float y[2][NC];
    const bool moved = __any_sync(0xffffffffu, over);
    if (moved) {  // move the references to the maximum, and the factors with them
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float top = fmaxf(fmaxf(lg[0][c], lg[1][c]), cs.ref[c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float down = ex2(cs.ref[c] - top);
        float xm = fmaxf(ex2(lg[0][c] - top) * sv[0], ex2(lg[1][c] - top) * sv[1]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
        const float vf = kYTop * pow2_below(fmaxf(xm, down * kYTop / cs.vf[c]));
        const float mul = down * vf / cs.vf[c];  // at most 1
        cs.ref[c] = top;
        cs.l[c] *= down;
        cs.m[c] *= down;
        cs.vf[c] = vf;
#pragma unroll
        for (int i2 = 0; i2 < L::MT; ++i2)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (kSplit || (e & 1) == c) acc[i2][e] *= mul;
      }
    }
    over = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float e = ex2(lg[h][c] - cs.ref[c]);
        cs.l[c] += e;
        cs.m[c] = fmaf(e, mv[h], cs.m[c]);
        y[h][c] = e * sv[h];
        over = over || y[h][c] * cs.vf[c] > kYMax;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float xm = fmaxf(fmaxf(y[0][c], y[1][c]), kYTop / cs.vf[c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
        const float vf = kYTop * pow2_below(xm), mul = vf / cs.vf[c];
        cs.vf[c] = vf;
#pragma unroll
        for (int i2 = 0; i2 < L::MT; ++i2)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (kSplit || (e & 1) == c) acc[i2][e] *= mul;
      }
    }
    uint32_t b0, b1;
    if constexpr (kSplit) {
      const float y0 = y[0][0] * cs.vf[0], y1 = y[1][0] * cs.vf[0];
      b0 = transposed(half2_bits(y0, y0 - __half2float(__float2half_rn(y0))));
      b1 = transposed(half2_bits(y1, y1 - __half2float(__float2half_rn(y1))));
    } else {
      b0 = transposed(half2_bits(y[0][0] * cs.vf[0], y[0][1] * cs.vf[1]));
      b1 = transposed(half2_bits(y[1][0] * cs.vf[0], y[1][1] * cs.vf[1]));
    }
    // output: product rows g, g + 8 are neighbouring elements of the lane's part of V
#pragma unroll
    for (int w = 0; w < L::VW; ++w) {
#pragma unroll
      for (int hh = 0; hh < (L::VB < 4 ? 1 : 2); ++hh) {
        const uint32_t sel = hh ? 0x7632 : 0x5410;
        const uint32_t a = __byte_perm(cur.v[0][w], cur.v[1][w], sel);
        const uint32_t b = __byte_perm(cur.v[2][w], cur.v[3][w], sel);
        if constexpr (BITS == 4) {
          mma16816(acc[4 * w + 2 * hh], a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu,
                   b & 0x00f000f0u, b0, b1);
          const uint32_t c = a >> 8, d = b >> 8;
          mma16816(acc[4 * w + 2 * hh + 1], c & 0x000f000fu, c & 0x00f000f0u, d & 0x000f000fu,
                   d & 0x00f000f0u, b0, b1);
        } else {
          mma16816(acc[2 * w + hh], a & 0x00ff00ffu, (a >> 8) & 0x00ff00ffu, b & 0x00ff00ffu,
                   (b >> 8) & 0x00ff00ffu, b0, b1);
        }
      }
    }
    cur = nxt;
    pos = npos;
  }

  // the warp's sums
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      cs.l[c] += __shfl_xor_sync(0xffffffffu, cs.l[c], o);
      cs.m[c] += __shfl_xor_sync(0xffffffffu, cs.m[c], o);
    }
    const int h = kSplit ? t : 2 * t + c;
    if (gq == 0) {
      sref[warp][h] = cs.ref[c];
      sl[warp][h] = cs.l[c];
    }
    const float back = 16777216.f / cs.vf[c];
#pragma unroll
    for (int i = 0; i < L::MT; ++i) {
      const int d = gq * (D / 8) + 2 * i;
      const float lo = kSplit ? acc[i][0] + acc[i][1] : acc[i][c];
      const float hi = kSplit ? acc[i][2] + acc[i][3] : acc[i][2 + c];
      so[warp][h][d] = fmaf(lo, back, cs.m[c]);
      so[warp][h][d + 1] = fmaf(hi, BITS == 4 ? back * 0.0625f : back, cs.m[c]);
    }
  }
  __syncthreads();
  // the CTA's
  for (int e = threadIdx.x; e < HC * D; e += kWarps * 32) {
    const int h = e / D, d = e % D;
    float top = sref[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sref[w][h]);
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sref[w][h] - top);
      o = fmaf(so[w][h][d], f, o);
      l = fmaf(sl[w][h], f, l);
    }
    so[0][h][d] = o;  // read by this thread alone
    if (d == 0) {
      cref[h] = top;
      cl[h] = l;
    }
  }
  if (csize > 1) cluster.sync();
  else __syncthreads();
  // the cluster's: each CTA a part of the elements
  for (int e = crank * kWarps * 32 + threadIdx.x; e < HC * D; e += csize * kWarps * 32) {
    const int h = e / D, d = e % D;
    if (h >= heads) continue;
    float top = kNone, o = 0.f, l = 0.f;
    if (csize == 1) {
      top = cref[h];
      o = so[0][h][d];
      l = cl[h];
    } else {
      for (int r = 0; r < csize; ++r) top = fmaxf(top, *cluster.map_shared_rank(&cref[h], r));
      for (int r = 0; r < csize; ++r) {
        const float f = ex2(*cluster.map_shared_rank(&cref[h], r) - top);
        o = fmaf(*cluster.map_shared_rank(&so[0][h][d], r), f, o);
        l = fmaf(*cluster.map_shared_rank(&cl[h], r), f, l);
      }
    }
    if (p.splits > 1) {
      float* w = p.part + ((item * p.splits + split) * HC + h) * (D + 2);
      w[d] = o;
      if (d == 0) {
        w[D] = top;
        w[D + 1] = l;
      }
    } else {
      const int64_t r = int64_t(un.row) * g.H + head0 + h;
      static_cast<T*>(p.out)[r * D + d] = T(l > 0.f || l != l ? o / l : 0.f);
      if (d == 0) p.lse[r] = l > 0.f || l != l ? (top + lg2(l)) * kLn2 : neg_inf();
    }
  }
  if (csize > 1) cluster.sync();  // nobody leaves while its sums are read
}

// joins the clusters of a unit: one thread an element
template <class T, int D>
__global__ void __launch_bounds__(256) cache_join_kernel(const AttnParams p, int hc) {
  const BlockGeom& g = p.c.g;
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int d = int(e % D);
  const int64_t q = e / D;  // query row * H + head
  if (q >= int64_t(g.U) * g.H) return;
  const int head = int(q % g.H), u = int(q / g.H);
  const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, u);
  if (x.s < 0) return;
  const int kh = head / g.G, in = head % g.G;
  const int64_t item = (int64_t(u) * g.Hkv + kh) * p.groups + in / hc;
  const float* w = p.part + (item * p.splits * hc + in % hc) * (D + 2);
  const int64_t step = int64_t(hc) * (D + 2);
  float top = kNone, o = 0.f, l = 0.f;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, w[s * step + D]);
  for (int s = 0; s < p.splits; ++s) {
    const float f = ex2(w[s * step + D] - top);
    o = fmaf(w[s * step + d], f, o);
    l = fmaf(w[s * step + D + 1], f, l);
  }
  static_cast<T*>(p.out)[q * D + d] = T(l > 0.f || l != l ? o / l : 0.f);
  if (d == 0) p.lse[q] = l > 0.f || l != l ? (top + lg2(l)) * kLn2 : neg_inf();
}

struct Shape {
  int hc, groups, cluster, splits;
};
Shape shape(const CacheParams& p, gattn_dtype dt, int max_keys, bool lists) {
  const BlockGeom& g = p.g;
  Shape s{};
  s.hc = dt == GATTN_F32 ? kCols / 2 : kCols;
  s.groups = (g.G + s.hc - 1) / s.hc;
  const int64_t items = int64_t(g.U) * g.Hkv * s.groups;
  const int64_t keys = lists ? std::min<int64_t>(int64_t(g.topk) * g.block, max_keys) : max_keys;
  const int64_t tiles = (keys + kTile - 1) / kTile;
  const int64_t slots = int64_t(sm_count()) * 2;
  int64_t n = 1;  // CTAs to an item: a power of two, with a tile at least for each warp
  while (items * n * 2 <= slots && n * 2 * kWarps <= tiles) n *= 2;
  s.cluster = int(std::min<int64_t>(n, kMaxCluster));
  s.splits = int(n / s.cluster);
  return s;
}

template <class T, int BITS, int D>
cudaError_t launch(const AttnParams& p, const Shape& s, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  const int64_t items = int64_t(p.c.g.U) * p.c.g.Hkv * s.groups;
  cfg.gridDim = dim3(unsigned(items * s.splits * s.cluster));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = unsigned(s.cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, cache_attn_kernel<T, BITS, D>, p);
  if (e != cudaSuccess || s.splits == 1) return e;
  const int64_t n = int64_t(p.c.g.U) * p.c.g.H * D;
  cache_join_kernel<T, D><<<unsigned((n + 255) / 256), 256, 0, st>>>(p, s.hc);
  return cudaGetLastError();
}

template <class T, int BITS>
cudaError_t by_width(const AttnParams& p, const Shape& s, cudaStream_t st) {
  if (p.c.g.D == 32) return launch<T, BITS, 32>(p, s, st);
  if (p.c.g.D == 64) return launch<T, BITS, 64>(p, s, st);
  return launch<T, BITS, 128>(p, s, st);
}

}  // namespace

size_t cache_fwd_workspace(const CacheParams& p, gattn_dtype dt, int max_keys, bool lists) {
  const Shape s = shape(p, dt, max_keys, lists);
  if (s.splits == 1) return 0;
  return size_t(p.g.U) * p.g.Hkv * s.groups * s.splits * s.hc * (p.g.D + 2) * 4;
}

gattn_status launch_cache_fwd(const CacheParams& c, gattn_dtype dt, int max_keys, const void* Q,
                              const int32_t* idx, void* out, float* lse, void* ws,
                              cudaStream_t st) {
  const Shape s = shape(c, dt, max_keys, idx != nullptr);
  AttnParams p{};
  p.c = c;
  p.Q = Q;
  p.idx = idx;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  p.groups = s.groups;
  p.splits = s.splits;
  p.max_keys = max_keys;
  if (int64_t(c.g.U) * c.g.Hkv * s.groups * s.splits * s.cluster > INT32_MAX) {
    set_error("gattn_cache_fwd: too many rows and heads");
    return GATTN_ERR_UNSUPPORTED;
  }
  const bool f32 = dt == GATTN_F32;
  const cudaError_t e = c.bits == 4 ? (f32 ? by_width<float, 4>(p, s, st)
                                           : by_width<__nv_bfloat16, 4>(p, s, st))
                                    : (f32 ? by_width<float, 8>(p, s, st)
                                           : by_width<__nv_bfloat16, 8>(p, s, st));
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("gattn_cache_fwd launch failed: %s", cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  return GATTN_OK;
}

}  // namespace gattn
