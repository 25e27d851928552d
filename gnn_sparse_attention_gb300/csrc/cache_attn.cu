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
// fifth of the legacy pipe.  S^T = K Q^T has rows of the cache as rows; P^T is
// turned by movmatrix into the right operand of O^T = V^T P^T.  A lane's elements
// of K and V are whole words of a row, since any order of the head's elements
// will do for K as long as q has the same, and for V it only names output rows.
//
// Precision.  q enters in fp16 after scaling each head by a power of two: exact
// for bf16, as a sum of two (two columns) for fp32.  p s enters in fp16 (11 bits,
// or as two for fp32), scaled by a power of two per column that follows its
// maximum.  Softmax statistics, m's terms and all sums are fp32.  The tensor cores
// align products by the operands' exponent fields, so a level at the bottom of the
// denormals loses the bits above it: K's are raised by three bits (lse of 128
// tokens off by 7e-8 instead of 1.2e-6, for 0.3 us of 62).  And sums about 0 round
// less than sums about q . middle level: scores start from minus that, with m + the
// middle's steps for m.  In fp32 both operands are moved about zero before their
// products (1024 + u in fp16 less 1024 + middle, one more instruction for two
// levels, 9 us of 62 where that was tried with bf16): out off by 2.3e-7, which was 2.3e-5.
//
// A warp takes steps of 32 rows (16 where a row has 128 bytes, 64 up to 32) through a ring of
// its own in shared memory, filled by cp.async two steps ahead, with its own running
// maximum and sum.  The maximum moves only when weights relative to it pass 2^6, seen in
// a step's sum of them, so a step needs one vote and no shuffles.
//
// Split.  The steps of all (query, key head) items are one line that is cut into
// equal stretches, one for each CTA that the GPU holds at a time, whatever the
// lengths of the sequences are: CTAs read them and find their stretch themselves.
// Items that lie within a stretch are finished there; of one that is cut, each CTA
// leaves its part in the workspace and a second kernel joins them.  While a CTA is at
// one item, a warp of it finds the next, whose first steps are fetched before the
// sums of the old one are joined.  Short items are a cluster's (or a CTA's) each and
// joined through its shared memory; see shape() for where that is better.
//
// Measured (32 heads of 128 on 8, 4 bits): 128 lists of 2,048 rows 55 us (285 MB, 5.2 TB/s), 8 whole
// caches of about 32,000 rows 59 us (5.2 TB/s; 6.3 at 128,000), 4 lists of 1,024 rows 8.1 us,
// all in captured graphs; in bf16 the first takes 172.  Half the issue slots and logic units are
// busy; what keeps short calls from the rate of long ones is fixed: 2.5 us to find the work, 4
// until the first rows are there, 2.4 for the join.  The first with fp32 queries 74 us (twice the columns,
// levels moved about zero), 64 heads on 8 62, 128 heads (a second pass) 110, D 64 39, in 8 bits 94.
// Queries of one sequence read it once each: 4 sequences of 6,000 rows with 5 each 32 us, of 4.1 that
// reading once would take.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"

namespace gattn {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThr = kWarps * 32;
constexpr int kCtas = 4;        // per SM
constexpr int kStages = 3;
constexpr int kMinSteps = 4;    // of a stretch: one for each warp
constexpr int kMaxCluster = 8;
constexpr int kMaxShared = 32;  // steps of a warp where items are not cut,
constexpr int kMaxSharedFew = 12;  // and where they fill less than a quarter of the GPU
constexpr float kOver = 64.f;   // weights relative to the running maximum: of a step's rows together
// A column whose scores stay within kStay (in log2) keeps its maximum when others move: a lane's 8 rows
// or fewer then weigh kOver or less.
constexpr float kStay = 3.f;
// Largest p s of a column in fp16: to [kYTop, 2 kYTop) when the factor is set, so that what is
// 2^-19 of it keeps its 11 bits; set again where a step could leave fp16's range.
constexpr float kYTop = 32.f, kYMax = 65504.f;

struct AttnParams {
  CacheParams c;
  const void* Q;
  const int32_t* idx;
  void* out;
  float* lse;
  float* part;   // [CTAs][2][heads][D + 4]: a stretch's first item if begun before, its last if cut
  int2* info;    // [items]: first CTA and CTAs of an item that is cut, (0, 0) for others
  int groups;    // column groups of a key head
  int ctas;      // stretches (0: a cluster for each item)
  int cluster;   // CTAs of that
  int max_keys;
};

template <int BITS, int D>
struct Lay {
  static constexpr int RB = D * BITS / 8;     // bytes of a row
  static constexpr int R = RB > 64 ? 16 : RB > 32 ? 32 : 64;  // rows of a step
  static constexpr int NT = R / 16;
  static constexpr int KW = RB / 16;          // words of a K row that a lane holds
  static constexpr int KL = KW < 4 ? KW : 4;  // ... in one load
  static constexpr int VB = RB / 8;           // bytes of a V row that a lane holds
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int MT = D / 16;           // 16-row tiles of the output
  static constexpr int QR = D / 8;            // registers of q per lane
  static constexpr int CP = R * RB / 512;     // 16-byte copies of a lane for K, and for V
  static constexpr int STAGE = R * (2 * RB + 8);
  static constexpr int RING = kStages * STAGE;  // bytes of a warp
};

__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^(127 - exponent) as a factor: x * pow2_below(x) is in [1, 2) for x in [2^-97, 2^(top - 126))
__device__ __forceinline__ float pow2_below(float x, int top) {
  const int e = (__float_as_uint(x) >> 23) & 255;
  return __uint_as_float(uint32_t(254 - clampi(e, 30, top)) << 23);
}
constexpr int kQTop = 253, kVTop = 224;  // of q: all of fp32; of p s: sums stay in it too
template <int N>
__device__ __forceinline__ void copy(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
// N bytes to shared memory, zeros where `in` is false (nothing is read then)
template <int N>
__device__ __forceinline__ void copy(uint32_t dst, const void* src, bool in) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src),
                 "r"(in ? 8 : 0) : "memory");
}

// Levels as fp16 numbers about zero: the bits `m` of x in the low bits of 1024, less 1024 and the
// middle level.  BITS 4: m names a nibble of each half, which counts 16 times if it is the upper one.
__device__ __forceinline__ uint32_t less(uint32_t x, uint32_t bias) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t nibble(uint32_t x) {
  return less((x & 0x000f000fu) | 0x64006400u, 0x64086408u);
}
__device__ __forceinline__ uint32_t nibble16(uint32_t x) {
  return less((x & 0x00f000f0u) | 0x64006400u, 0x64806480u);
}
// bytes as they stand in the halves of x
__device__ __forceinline__ uint32_t byte(uint32_t x) {
  return less((x & 0x00ff00ffu) | 0x64006400u, 0x64806480u);
}

// Row of a tile that stands in product row r (r < 8; r + 8 likewise): product
// rows 2t, 2t + 1 are rows t, 4 + t, so that a warp's load of V covers four whole rows.
__device__ __forceinline__ int tile_row(int r) { return (r >> 1) + 4 * (r & 1); }

// Byte of 16-byte chunk `ch` of row `row` in a stage.  The lanes that shared memory
// serves together (a quarter of a warp for 16 bytes, half of one for 8) read rows a, a + 4
// of K and four rows of V; the exclusive-ors put those in different banks.
template <int RB>
__device__ __forceinline__ int k_byte(int row, int ch) {
  if (RB == 128) ch ^= ((row >> 2) & 1) << 2;
  if (RB == 64) row ^= (row >> 2) & 1;
  if (RB == 32) row ^= ((row >> 2) & 1) << 1;
  return row * RB + ch * 16;
}
template <int RB>
__device__ __forceinline__ int v_byte(int row, int ch) {
  if (RB == 128) ch ^= (row & 3) << 1;
  if (RB == 64) ch ^= ((row >> 1) & 1) << 1;
  return row * RB + ch * 16;
}

// What weights are taken relative to where the greatest score is `top`: -inf stands for no score, and
// finite scores may be as low as fp32 goes.
__device__ __forceinline__ float base_of(float top) { return top == neg_inf() ? 0.f : top; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void store4(float* to, float4 x) { *reinterpret_cast<float4*>(to) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* to, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                             *reinterpret_cast<const uint32_t*>(&b));
}

// A query row: where its sequence's rows lie in the cache, how many of them it
// may see, and the steps that takes (at least one; none for rows of no sequence).
struct Row {
  int beg, len, limit, steps;
};
template <int R>
__device__ __forceinline__ Row row_at(const AttnParams& p, int u) {
  const BlockGeom& g = p.c.g;
  // with one row a sequence, as in serving, row u is sequence u: looked at first, since a search
  // is a chain of loads
  int s = min(u, g.S - 1);
  const int b = clampi(g.seq_q[s], 0, g.Nq), e = clampi(g.seq_q[s + 1], b, g.Nq);
  Span sp = span_k(g, s);
  int i = u - b, n = e - b;
  Row r{};
  if (u < b || u >= e) {
    const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, u);
    if (x.s < 0) return r;
    sp = span_k(g, x.s);
    i = x.i;
    n = x.n;
  }
  r.beg = sp.beg;
  r.len = sp.len;
  r.limit = min(g.causal ? clampi(i + sp.len - n + 1, 0, sp.len) : sp.len, p.max_keys);
  const int keys = p.idx ? min(r.limit, g.topk * g.block) : r.limit;
  r.steps = max((keys + R - 1) / R, 1);
  return r;
}

// What a CTA works on: steps [s0, s1) of the `steps` of an item (row u, hi: key head and column
// group).  `keys` rows are seen, listed in ids or all; none left: steps = 0.
struct Seg {
  int u, hi, s0, s1, steps, keys, beg;
  int ids[kBlkMaxTopk];
};

// NC heads to a lane's two columns of a product.  With two, a group is 8 heads.  With one it is 4:
// in fp32 the head's two parts, in bf16 the second column is empty, which spares a group of up to
// 4 heads the softmax of columns that nobody has.
template <class T, int BITS, int D, int NC>
__global__ void __launch_bounds__(kThr, kCtas) cache_attn_kernel(const AttnParams p) {
  using L = Lay<BITS, D>;
  constexpr int RB = L::RB, R = L::R, NT = L::NT;
  constexpr bool kSplit = sizeof(T) == 4;  // fp32: a head is two columns
  constexpr int HC = 4 * NC;               // heads of a column group
  constexpr float kMid = BITS == 4 ? 8.f : 128.f;  // middle level
  static_assert(NC == 1 || !kSplit, "");
  static_assert(HC * D * 4 <= L::STAGE, "a warp's sums take the place of one stage, beside the next item's copies");
  static_assert(2 * NT * 8.f <= kOver, "a lane's rows, each of weight 2^kStay");
  extern __shared__ __align__(128) uint8_t ring[];  // [warp][stage]: K, V, par of R rows
  __shared__ Seg segs[2];                           // this one and the next
  __shared__ float sref[kWarps][HC], sl[kWarps][HC], sw[kWarps][HC];
  __shared__ int so_at[kWarps];
  __shared__ int64_t scan[kWarps];
  __shared__ int64_t cur_at, cur_end;  // the stretch, relative to row cur_u's first step
  __shared__ int cur_u;
  const BlockGeom& g = p.c.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
  const int heads_of = g.Hkv * p.groups;  // items of a query row
  const int rank = p.ctas ? 0 : blockIdx.x % p.cluster;
  const int wide = kWarps * (p.ctas ? 1 : p.cluster);  // warps that share an item's steps

  // where the stretch begins and ends, on the line of all items' steps
  int64_t per = 0;
  cudaTriggerProgrammaticLaunchCompletion();  // the join may be launched; it waits for this grid
  if (p.ctas) {
    const int k = (g.U + kThr - 1) / kThr, u0 = threadIdx.x * k, u1 = min(u0 + k, g.U);
    int64_t mine = 0;
    for (int i = u0; i < u1; ++i) mine += row_at<R>(p, i).steps;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int64_t total = 0, before = x - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    total *= heads_of;
    before *= heads_of;
    mine *= heads_of;
    per = max((total + p.ctas - 1) / p.ctas, int64_t(kMinSteps));
    const int64_t at = per * blockIdx.x, end = min(at + per, total);
    if (at >= end) return;
    if (at >= before && at < before + mine) {  // one thread
      int i = u0;
      for (; i + 1 < u1; ++i) {
        const int64_t n = int64_t(row_at<R>(p, i).steps) * heads_of;
        if (at < before + n) break;
        before += n;
      }
      cur_u = i;
      cur_at = at - before;
      cur_end = end - before;
    }
    __syncthreads();
  }

  // The next stretch of an item, by the first warp.
  const auto next = [&](Seg& to, bool first) {
    int u, hi = 0, s0 = 0, s1 = 0;
    Row r{};
    if (p.ctas) {
      int64_t at = cur_at, end = cur_end;
      u = cur_u;
      while (at < end && u < g.U) {
        r = row_at<R>(p, u);
        const int64_t row_steps = int64_t(r.steps) * heads_of;
        if (at < row_steps) break;
        at -= row_steps;
        end -= row_steps;
        ++u;
      }
      if (at < end && u < g.U) {
        hi = int(at / r.steps);
        s0 = int(at - int64_t(hi) * r.steps);
        s1 = int(min(int64_t(r.steps), s0 + (end - at)));
      } else {
        r.steps = 0;
      }
      __syncwarp();
      if (lane == 0) {
        cur_u = u;
        cur_at = at + (s1 - s0);
        cur_end = end;
      }
    } else {
      const int item = blockIdx.x / p.cluster;
      u = item / heads_of;
      hi = item % heads_of;
      if (first) r = row_at<R>(p, u);
      s1 = r.steps;
    }
    int keys = r.limit;
    if (p.idx && r.steps) {
      const int nb = (r.len + g.block - 1) / g.block;
      const int n = block_list(
          p.idx + int64_t(u) * g.is_u + int64_t(hi / p.groups) * g.is_h, g.topk, nb, to.ids);
      keys = list_keys(to.ids, n, g.block, r.limit);
    }
    if (lane == 0) {
      to.u = u;
      to.hi = hi;
      to.s0 = s0;
      to.s1 = s1;
      to.steps = r.steps;
      to.keys = keys;
      to.beg = r.beg;
    }
    __syncwarp();
  };

  const uint32_t my_ring = uint32_t(__cvta_generic_to_shared(ring)) + warp * L::RING;
  const uint8_t* my_stage = ring + warp * L::RING;
  const int lb = 31 - __clz(g.block);
  // where a lane's copies go: the exclusive-ors hang on the lane alone, but for rows of 128 bytes
  const int kc = k_byte<RB>(lane * 16 / RB, lane * 16 % RB / 16);
  const int vc = R * RB + v_byte<RB>(lane * 16 / RB, lane * 16 % RB / 16);
  // what a lane reads of a stage
  const int ko = k_byte<RB>(tile_row(gq), t * L::KL * 4 / 16) + t * L::KL * 4 % 16;
  const int vo = R * RB + v_byte<RB>(t, gq * L::VB / 16) + gq * L::VB % 16;
  const int po = 2 * R * RB + tile_row(gq) * 8;

  const Seg* seg = segs;
  const uint8_t *kb, *vb;  // the item's rows
  const uint2* pb;
  int keys, steps;
  const auto open = [&]() {
    const int64_t row0 = int64_t(seg->hi / p.groups) * g.Nk + seg->beg;
    kb = p.c.k + row0 * RB;
    vb = p.c.v + row0 * RB;
    pb = p.c.par + row0;
    keys = seg->keys;
    steps = min(seg->s1, (keys + R - 1) / R);
  };
  // position of row `i` of the item's rows; rows of a tile lie side by side
  const auto tile_pos = [&](int i) {
    return p.idx ? (seg->ids[i >> lb] << lb) + (i & (g.block - 1)) : i;
  };
  const auto fetch = [&](int step, int to) {
    const uint32_t dst = my_ring + to * L::STAGE;
    if ((step + 1) * R <= keys && step < steps) {
      int pos[NT];  // where the tile's rows lie, less those before it in the step
#pragma unroll
      for (int h = 0; h < NT; ++h) pos[h] = tile_pos(step * R + 16 * h) - 16 * h;
#pragma unroll
      for (int j = 0; j < L::CP; ++j) {
        const int h = RB == 16 ? 2 * j : j * 512 / RB / 16;
        const int at = RB == 16 && lane >= 16 ? pos[h + 1 < NT ? h + 1 : h] : pos[h];
        const int64_t from = int64_t(at) * RB + lane * 16 + j * 512;
        copy<16>(dst + (kc ^ (RB == 128 ? (j & 1) * 64 : 0)) + j * 512, kb + from);
        copy<16>(dst + vc + j * 512, vb + from);
      }
#pragma unroll
      for (int j = 0; j < (R + 31) / 32; ++j) {
        const int at = lane < 16 ? pos[2 * j] : pos[2 * j + 1 < NT ? 2 * j + 1 : 2 * j];
        if (R >= 32 || lane < R)
          copy<8>(dst + 2 * R * RB + lane * 8 + j * 256, pb + at + lane + 32 * j);
      }
    } else if (step < steps) {  // the last one: zeros behind the rows that the query sees
#pragma unroll 1
      for (int j = 0; j < L::CP; ++j) {
        const int c = j * 512 + lane * 16, row = c / RB, ch = c % RB / 16;
        const int i = step * R + row;
        const bool in = i < keys;
        const int64_t from = in ? int64_t(tile_pos(i)) * RB + ch * 16 : 0;
        copy<16>(dst + k_byte<RB>(row, ch), kb + from, in);
        copy<16>(dst + R * RB + v_byte<RB>(row, ch), vb + from, in);
      }
      for (int r = lane; r < R; r += 32) {
        const int i = step * R + r;
        copy<8>(dst + 2 * R * RB + r * 8, pb + (i < keys ? tile_pos(i) : 0), i < keys);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  const auto follow = [&](int stage) { return stage + 1 == kStages ? 0 : stage + 1; };

  if (warp == 0) next(segs[0], true);
  __syncthreads();
  if (segs[0].steps == 0) {  // a row of no sequence
    if (p.ctas == 0 && p.cluster > 1) {
      // If offsets change meanwhile, others of the cluster may have seen one: they read this
      // CTA's sums, so it stays, with none.
      if (threadIdx.x < HC) {
        sref[0][threadIdx.x] = neg_inf();
        sl[0][threadIdx.x] = 0.f;
      }
      if (threadIdx.x == 0) so_at[0] = 0;
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      cluster.sync();
    }
    return;
  }
  open();
  int stage = 0;
  fetch(seg->s0 + rank * kWarps + warp, 0);
  fetch(seg->s0 + rank * kWarps + warp + wide, 1);

  for (;;) {
    if (warp == 0) next(segs[seg == segs], false);
    const int kh = seg->hi / p.groups, cgrp = seg->hi % p.groups;
    const int head0 = kh * g.G + cgrp * HC, heads = min(HC, g.G - cgrp * HC);
    // q of this lane's column, scaled to fp16's range, in the order of the words of a K row
    uint32_t qf[L::QR];
    float qmul[NC], qsum[NC], qmid[NC];  // of the lane's heads
    {
      const int hc = NC == 1 ? gq >> 1 : gq;
      const bool on = hc < heads && (NC == 2 || kSplit || !(gq & 1));
      const T* q = static_cast<const T*>(p.Q) + (int64_t(seg->u) * g.H + head0 + (on ? hc : 0)) * D;
      constexpr int PW = 32 / BITS;           // elements of a word
      constexpr int RUN = L::KL * PW;         // neighbouring elements of a lane
      constexpr int VE = 16 / int(sizeof(T));
      float f[L::KW * PW], top = 0.f;
#pragma unroll
      for (int c = 0; c < L::KW / L::KL; ++c)
#pragma unroll
        for (int i = 0; i < RUN; i += VE) {
          const uint4 x = *reinterpret_cast<const uint4*>(q + c * (64 * 8 / BITS) + t * RUN + i);
          const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
          for (int z = 0; z < VE; ++z) f[c * RUN + i + z] = to_f32(e[z]);
        }
#pragma unroll
      for (int i = 0; i < L::KW * PW; ++i) top = fmaxf(top, fabsf(f[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float scale = pow2_below(top, kQTop) * 8192.f;  // largest element to [2^13, 2^14)
      const float up = on ? scale : 0.f, up16 = up * 0.0625f;
#pragma unroll
      for (int w = 0; w < L::KW; ++w)
#pragma unroll
        for (int i = 0; i < PW; i += 4) {
          // 4 bits, by the masked halves of the word: (0, 4) and (1, 5), then (2, 6) and (3, 7);
          // 8 bits: (0, 2) and (1, 3).  Upper nibbles count 16 times.
          float x[4];
          if constexpr (BITS == 4) {
            x[0] = f[w * PW + i / 2] * up; x[1] = f[w * PW + 4 + i / 2] * up;
            x[2] = f[w * PW + i / 2 + 1] * up16; x[3] = f[w * PW + 4 + i / 2 + 1] * up16;
          } else {
            x[0] = f[w * PW] * up; x[1] = f[w * PW + 2] * up;
            x[2] = f[w * PW + 1] * up; x[3] = f[w * PW + 3] * up;
          }
          if (kSplit && (gq & 1)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] -= __half2float(__float2half_rn(x[e]));
          }
          const int r = (w * PW + i) / 2;
          qf[r] = half2_bits(x[0], x[1]);
          qf[r + 1] = half2_bits(x[2], x[3]);
        }
      // columns 2t, 2t + 1 of a product belong to the lanes with gq = 2t, 2t + 1; the sum of q is
      // its product with levels of 1
      const float mul = g.qmul * (kSplit ? 1.f : 0x1p21f) / scale;
      float one[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < L::QR; r += 2) {
        constexpr uint32_t kOne = kSplit ? 0x3c003c00u : 0x00080008u;
        constexpr uint32_t kUp = BITS == 8 ? kOne : kSplit ? 0x4c004c00u : 0x00800080u;
        mma16816(one, kOne, kOne, kUp, kUp, qf[r], qf[r + 1]);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float x = kSplit ? one[0] + one[1] : one[c];
        qmul[c] = __shfl_sync(0xffffffffu, mul, (2 * t + c) * 4);
        qsum[c] = x * qmul[c];
        qmid[c] = -kMid * x;
      }
    }

    float acc[L::MT][4];
#pragma unroll
    for (int i = 0; i < L::MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float ref[NC], sum[NC], msum[NC], vf[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      ref[c] = 0.f;
      sum[c] = msum[c] = 0.f;
      vf[c] = 1.f;
    }

    bool fresh = true;  // no step so far; each has a row that is seen
    for (int step = seg->s0 + rank * kWarps + warp; step < steps; step += wide) {
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // all lanes' copies are here, and the stage to be filled has been read
      fetch(step + 2 * wide, stage == 0 ? kStages - 1 : stage - 1);
      const uint8_t* st = my_stage + stage * L::STAGE;
      stage = follow(stage);
      // scores relative to the running maximum, in log2
      float x[NT][2][NC], vs[NT][2], vm[NT][2];
      bool over;
      float s4[NT][4];
      uint32_t ka[NT][2][L::KW];
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        s4[h][0] = s4[h][1] = s4[h][2] = s4[h][3] = 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int c = 0; c < L::KW / L::KL; ++c) {
            const uint8_t* a = st + (ko ^ (c * 64)) + (16 * h + 8 * q) * RB;
            if constexpr (L::KL == 4) {
              const uint4 w = *reinterpret_cast<const uint4*>(a);
              ka[h][q][4 * c] = w.x; ka[h][q][4 * c + 1] = w.y;
              ka[h][q][4 * c + 2] = w.z; ka[h][q][4 * c + 3] = w.w;
            } else if constexpr (L::KL == 2) {
              const uint2 w = *reinterpret_cast<const uint2*>(a);
              ka[h][q][0] = w.x; ka[h][q][1] = w.y;
            } else {
              ka[h][q][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
      }
#pragma unroll
      for (int w = 0; w < L::KW; ++w)
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          const uint32_t a = ka[h][0][w], b = ka[h][1][w];
          const uint32_t* const q = qf + w * (L::QR / L::KW);
          if constexpr (kSplit && BITS == 4) {
            mma16816(s4[h], nibble(a), nibble(b), nibble16(a), nibble16(b), q[0], q[1]);
            const uint32_t c = a >> 8, d = b >> 8;
            mma16816(s4[h], nibble(c), nibble(d), nibble16(c), nibble16(d), q[2], q[3]);
          } else if constexpr (kSplit) {
            mma16816(s4[h], byte(a), byte(b), byte(a >> 8), byte(b >> 8), q[0], q[1]);
          } else {
            if (w == 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) s4[h][e] = NC == 2 || e % 2 == 0 ? qmid[NC == 2 ? e % 2 : 0] : 0.f;
            }
            if constexpr (BITS == 4) {
              const uint32_t c = a << 3, d = b << 3, e = a >> 5, f = b >> 5;
              mma16816(s4[h], c & 0x00780078u, d & 0x00780078u, c & 0x07800780u, d & 0x07800780u,
                       q[0], q[1]);
              mma16816(s4[h], e & 0x00780078u, f & 0x00780078u, e & 0x07800780u, f & 0x07800780u,
                       q[2], q[3]);
            } else {
              const uint32_t c = a << 3, d = b << 3, e = a >> 5, f = b >> 5;
              mma16816(s4[h], c & 0x07f807f8u, d & 0x07f807f8u, e & 0x07f807f8u, f & 0x07f807f8u,
                       q[0], q[1]);
            }
          }
        }
#pragma unroll
      for (int h = 0; h < NT; ++h) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint2 par = *reinterpret_cast<const uint2*>(st + po + (16 * h + 8 * q) * 8);
          const float mk = __uint_as_float(par.x << 16), sk = __uint_as_float(par.x & 0xffff0000u);
          vs[h][q] = __uint_as_float(par.y & 0xffff0000u);
          vm[h][q] = __uint_as_float(par.y << 16);
          if (kSplit) vm[h][q] = fmaf(kMid, vs[h][q], vm[h][q]);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float dot = kSplit ? s4[h][2 * q] + s4[h][2 * q + 1] : s4[h][2 * q + c];
            x[h][q][c] = fmaf(dot * qmul[c], sk, fmaf(fmaf(kMid, sk, mk), qsum[c], -ref[c]));
          }
        }
      }
      if ((step + 1) * R > keys) {  // rows behind the last that the query sees
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (step * R + 16 * h + 8 * q + tile_row(gq) >= keys) {
#pragma unroll
              for (int c = 0; c < NC; ++c) x[h][q][c] = neg_inf();
            }
      }
      // Weights and p s.  A score beyond kOver shows in the step's sum of weights, a p s beyond fp16 in
      // theirs.
      float e[NT][2][NC], y[NT][2][NC];
      float step_sum[NC];
      const auto weigh = [&]() {
        bool far = false;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float es = 0.f, ys = 0.f;
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              e[h][q][c] = ex2(x[h][q][c]);
              // in this order a weight of 0 gives 0 whatever the factor makes of the step alone
              y[h][q][c] = e[h][q][c] * vs[h][q] * vf[c];
              es += e[h][q][c];
              ys += y[h][q][c];
            }
          far = far || es > kOver || ys > kYMax;
          step_sum[c] = es;
        }
        return far;
      };
      over = weigh() || fresh;
      if (__any_sync(0xffffffffu, over)) {
        // references to the maxima, and the factors of p s with them
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float top = fresh ? neg_inf() : 0.f;
#pragma unroll
          for (int h = 0; h < NT; ++h) top = fmaxf(top, fmaxf(x[h][0][c], x[h][1][c]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (top == neg_inf() || (!fresh && top <= kStay)) top = 0.f;  // -inf: no score is a number
          float xm = 0.f;
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              x[h][q][c] -= top;
              xm = fmaxf(xm, ex2(x[h][q][c]) * vs[h][q]);
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
          const float down = fresh ? 0.f : ex2(-top);
          const float f = kYTop * pow2_below(fmaxf(xm, down * kYTop / vf[c]), kVTop);
          // Below 2, and 1 or less for a column that stays.  One that moves loses 2^kStay at least, which
          // vf gains besides mul: vf is at its limit after 49 moves, before acc grows by 2^49 (it starts
          // below 2^23 for a row).
          const float mul = down * f / vf[c];
          ref[c] += top;
          sum[c] *= down;
          msum[c] *= down;
          vf[c] = f;
#pragma unroll
          for (int i = 0; i < L::MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (NC == 1 || (e & 1) == c) acc[i][e] *= mul;
        }
        fresh = false;
        weigh();
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) sum[c] += step_sum[c];
#pragma unroll
      for (int h = 0; h < NT; ++h) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int c = 0; c < NC; ++c) msum[c] = fmaf(e[h][q][c], vm[h][q], msum[c]);
        uint32_t b0, b1;
        if constexpr (kSplit) {
          b0 = transposed(half2_bits(y[h][0][0], y[h][0][0] - __half2float(__float2half_rn(y[h][0][0]))));
          b1 = transposed(half2_bits(y[h][1][0], y[h][1][0] - __half2float(__float2half_rn(y[h][1][0]))));
        } else {
          b0 = transposed(half2_bits(y[h][0][0], NC == 2 ? y[h][0][NC - 1] : 0.f));
          b1 = transposed(half2_bits(y[h][1][0], NC == 2 ? y[h][1][NC - 1] : 0.f));
        }
        uint32_t va[4][L::VW];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint8_t* a = st + vo + (16 * h + 4 * q) * RB;
          if constexpr (L::VB == 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(a);
            va[q][0] = w.x; va[q][1] = w.y; va[q][2] = w.z; va[q][3] = w.w;
          } else if constexpr (L::VB == 8) {
            const uint2 w = *reinterpret_cast<const uint2*>(a);
            va[q][0] = w.x; va[q][1] = w.y;
          } else if constexpr (L::VB == 4) {
            va[q][0] = *reinterpret_cast<const uint32_t*>(a);
          } else {
            va[q][0] = *reinterpret_cast<const uint16_t*>(a);
          }
        }
        // output: product rows g, g + 8 are neighbouring elements of the lane's part of V
#pragma unroll
        for (int w = 0; w < L::VW; ++w)
#pragma unroll
          for (int hh = 0; hh < (L::VB < 4 ? 1 : 2); ++hh) {
            const uint32_t sel = hh ? 0x7632 : 0x5410;
            const uint32_t a = __byte_perm(va[0][w], va[1][w], sel);
            const uint32_t b = __byte_perm(va[2][w], va[3][w], sel);
            if constexpr (BITS == 4) {
              const uint32_t c = a >> 8, d = b >> 8;
              float *o = acc[4 * w + 2 * hh], *o2 = acc[4 * w + 2 * hh + 1];
              if constexpr (kSplit) {
                mma16816(o, nibble(a), nibble16(a), nibble(b), nibble16(b), b0, b1);
                mma16816(o2, nibble(c), nibble16(c), nibble(d), nibble16(d), b0, b1);
              } else {
                mma16816(o, a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu, b & 0x00f000f0u, b0, b1);
                mma16816(o2, c & 0x000f000fu, c & 0x00f000f0u, d & 0x000f000fu, d & 0x00f000f0u, b0, b1);
              }
            } else if constexpr (kSplit) {
              mma16816(acc[2 * w + hh], byte(a), byte(a >> 8), byte(b), byte(b >> 8), b0, b1);
            } else {
              mma16816(acc[2 * w + hh], a & 0x00ff00ffu, (a >> 8) & 0x00ff00ffu, b & 0x00ff00ffu,
                       (b >> 8) & 0x00ff00ffu, b0, b1);
            }
          }
      }
    }

    // The warp's sums, in the stage that the next item's first steps leave free.  No copy is under
    // way: there were none beyond the last step.
    __syncwarp();
    const int free_at = warp * L::RING + follow(follow(stage)) * L::STAGE;
    float* so = reinterpret_cast<float*>(ring + free_at);  // [HC][D]
    if (lane == 0) so_at[warp] = free_at;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], o);
        msum[c] += __shfl_xor_sync(0xffffffffu, msum[c], o);
      }
      const int h = NC * t + c;
      if (gq == 0) {
        sref[warp][h] = fresh ? neg_inf() : ref[c];
        sl[warp][h] = sum[c];
      }
      const float back = (kSplit ? 1.f : 16777216.f) / vf[c];
#pragma unroll
      for (int i = 0; i < L::MT; ++i) {
        const float lo = kSplit ? acc[i][0] + acc[i][1] : acc[i][c];
        const float up = kSplit ? acc[i][2] + acc[i][3] : acc[i][2 + c];
        *reinterpret_cast<float2*>(so + h * D + gq * (D / 8) + 2 * i) =
            make_float2(fmaf(lo, back, msum[c]),
                        fmaf(up, BITS == 4 ? back * 0.0625f : back, msum[c]));
      }
    }
    __syncthreads();
    const Seg* const done = seg;
    const bool more = segs[seg == segs].steps != 0;
    if (more) {
      seg = segs + (seg == segs);
      open();
      fetch(seg->s0 + warp, stage);
      fetch(seg->s0 + warp + kWarps, follow(stage));
    }
    // the CTA's: finished, or its part of the item
    const bool cut = done->s1 - done->s0 < done->steps;
    const bool shared = p.ctas == 0 && p.cluster > 1;
    const int64_t out0 = int64_t(done->u) * g.H + head0;
    float* part = p.part + (int64_t(blockIdx.x) * 2 + (done->s0 == 0)) * HC * (D + 4);
    if (threadIdx.x < HC) {
      const int h = threadIdx.x;
      float top = sref[0][h], l = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sref[w][h]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(sref[w][h] - base_of(top));
        l = fmaf(sl[w][h], f, l);
        sw[w][h] = f;
      }
      // what a finished element is multiplied by, and the statistics
      const bool some = l > 0.f || l != l;
      if (shared) {
        sref[0][h] = top;
        sl[0][h] = l;
      } else if (cut) {
        if (h < heads) *reinterpret_cast<float2*>(part + h * (D + 4) + D) = make_float2(top, l);
      } else {
        const float r = some ? 1.f / l : 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sw[w][h] *= r;
        if (h < heads) p.lse[out0 + h] = some ? (top + lg2(l)) * kLn2 : neg_inf();
      }
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < heads * D; e += kThr * 4) {
      const int h = e / D, d = e % D;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(ring + so_at[w] + e * 4);
        const float f = sw[w][h];
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
      }
      if (shared) *reinterpret_cast<float4*>(ring + so_at[0] + e * 4) = o;  // read by this thread alone
      else if (cut) *reinterpret_cast<float4*>(part + h * (D + 4) + d) = o;
      else store4(static_cast<T*>(p.out) + (out0 + h) * D + d, o);
    }
    if (shared) {  // the cluster's: each CTA a part of the elements
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      for (int e = (rank * kThr + threadIdx.x) * 4; e < heads * D; e += p.cluster * kThr * 4) {
        const int h = e / D, d = e % D;
        float top = neg_inf(), l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < p.cluster; ++r)
          top = fmaxf(top, *cluster.map_shared_rank(&sref[0][h], r));
        for (int r = 0; r < p.cluster; ++r) {
          const float f = ex2(*cluster.map_shared_rank(&sref[0][h], r) - base_of(top));
          const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(
              ring + *cluster.map_shared_rank(&so_at[0], r) + e * 4, r));
          o.x = fmaf(x.x, f, o.x);
          o.y = fmaf(x.y, f, o.y);
          o.z = fmaf(x.z, f, o.z);
          o.w = fmaf(x.w, f, o.w);
          l = fmaf(*cluster.map_shared_rank(&sl[0][h], r), f, l);
        }
        const bool some = l > 0.f || l != l;
        const float r = some ? 1.f / l : 0.f;
        store4(static_cast<T*>(p.out) + (out0 + h) * D + d,
               make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
        if (d == 0) p.lse[out0 + h] = some ? (top + lg2(l)) * kLn2 : neg_inf();
      }
      cluster.sync();  // nobody leaves while its sums are read
    }
    if (p.ctas && threadIdx.x == 0 && done->s0 == 0)
      p.info[int64_t(done->u) * heads_of + done->hi] =
          cut ? make_int2(blockIdx.x, 1 + min(int((done->steps - done->s1 + per - 1) / per),
                                              p.ctas - 1 - int(blockIdx.x)))
              : make_int2(0, 0);
    if (!more) return;
    __syncthreads();  // statistics, sums and the old item have been read
  }
}

// Joins an item that was cut.  A thread has four elements; the threads that the
// block has more than these share the parts.
template <class T, int D>
__global__ void __launch_bounds__(256) cache_join_kernel(const AttnParams p, int hc) {
  __shared__ float4 so[256];
  __shared__ float sr[256], sl[256];
  const BlockGeom& g = p.c.g;
  const int heads_of = g.Hkv * p.groups;
  const int u = blockIdx.x / heads_of, hi = blockIdx.x % heads_of;
  const int cgrp = hi % p.groups, kh = hi / p.groups;
  const int heads = min(hc, g.G - cgrp * hc);
  const int quads = heads * (D / 4);                        // of the item
  const int mine = (quads + gridDim.y - 1) / gridDim.y;     // of this block: at most 256
  const int q = blockIdx.y * mine + threadIdx.x % mine, grp = threadIdx.x / mine, ng = 256 / mine;
  const bool live = seq_row(g.seq_q, g.S, g.Nq, u).s >= 0;
  cudaGridDependencySynchronize();  // the parts are there
  int2 in = live ? p.info[blockIdx.x] : make_int2(0, 0);
  // parts that exist, also where offsets changed meanwhile and nobody wrote the item's entry
  in.x = clampi(in.x, 0, p.ctas - 1);
  in.y = clampi(in.y, 0, p.ctas - in.x);
  if (in.y == 0) return;
  const int h = q / (D / 4), d = q % (D / 4) * 4;
  float top = neg_inf(), l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (q < quads && grp < ng) {
#pragma unroll 4
    for (int i = grp; i < in.y; i += ng) {
      // part i: the first CTA's second slot, then the first slots of those that follow
      const float* w = p.part + (((int64_t(in.x) + i) * 2 + (i == 0)) * hc + h) * (D + 4);
      const float4 x = *reinterpret_cast<const float4*>(w + d);
      const float2 st = *reinterpret_cast<const float2*>(w + D);
      const float m = fmaxf(top, st.x), f0 = ex2(top - base_of(m)), f1 = ex2(st.x - base_of(m));
      o.x = fmaf(o.x, f0, x.x * f1);
      o.y = fmaf(o.y, f0, x.y * f1);
      o.z = fmaf(o.z, f0, x.z * f1);
      o.w = fmaf(o.w, f0, x.w * f1);
      l = fmaf(l, f0, st.y * f1);
      top = m;
    }
  }
  so[threadIdx.x] = o;
  sr[threadIdx.x] = top;
  sl[threadIdx.x] = l;
  __syncthreads();
  if (grp > 0 || q >= quads) return;
  for (int i = 1; i < ng; ++i) {
    const int x = threadIdx.x + i * mine;
    const float m = fmaxf(top, sr[x]), f0 = ex2(top - base_of(m)), f1 = ex2(sr[x] - base_of(m));
    o.x = fmaf(o.x, f0, so[x].x * f1);
    o.y = fmaf(o.y, f0, so[x].y * f1);
    o.z = fmaf(o.z, f0, so[x].z * f1);
    o.w = fmaf(o.w, f0, so[x].w * f1);
    l = fmaf(l, f0, sl[x] * f1);
    top = m;
  }
  const bool some = l > 0.f || l != l;
  const float r = some ? 1.f / l : 0.f;
  const int64_t row = int64_t(u) * g.H + kh * g.G + cgrp * hc + h;
  store4(static_cast<T*>(p.out) + row * D + d, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
  if (d == 0) p.lse[row] = some ? (top + lg2(l)) * kLn2 : neg_inf();
}

struct Shape {
  int hc, groups;
  int64_t items;
  int ctas, cluster;  // see AttnParams
  size_t bytes;       // of the workspace: parts, then the items' table
};
Shape shape(const CacheParams& p, gattn_dtype dt, int max_keys, bool lists) {
  const BlockGeom& g = p.g;
  Shape s{};
  s.hc = dt == GATTN_F32 || g.G <= 4 ? 4 : 8;
  s.groups = (g.G + s.hc - 1) / s.hc;
  s.items = int64_t(g.U) * g.Hkv * s.groups;
  s.cluster = 1;
  const int64_t keys = lists ? std::min<int64_t>(int64_t(g.topk) * g.block, max_keys) : max_keys;
  const int row = g.D * p.bits / 8, rows = row > 64 ? 16 : row > 32 ? 32 : 64;  // Lay::R
  const int64_t steps = std::max<int64_t>((keys + rows - 1) / rows, 1);
  const int64_t slots = int64_t(sm_count()) * kCtas;
  // A cluster for each item, of as many CTAs as fill the GPU, where that leaves a warp at most
  // kMaxShared steps (or where there are so many items that the last to run weigh little); else
  // stretches.  Stretches keep long sequences of unlike lengths from waiting for the longest and use
  // all SMs for few; but each CTA reads all lengths, goes through more items, and a second kernel
  // joins.  Measured, us by clusters / by stretches (32 heads on 8; steps of 32 rows at D 128 with 4 bits
  // and D 64 with 8, of 64 at D 64 with 4 bits, of 16 at D 128 with 8):
  //                               D 128, 4 bits   8 bits          D 64, 4 bits    8 bits          D 128, 4 bits, fp32
  //   128 lists of 2,048 rows     55.0 / 62.4     93.0 / 100      39.0 / 45.1     54.6 / 57.4     73.3 / 82.0
  //   of 4,096 rows               97.0 / 105      172 / 183       61.7 / 68.6     95.7 / 101      131 / 140
  //   of 8,192 rows               179 / 188       329 / 345       109 / 117       177 / 187       246 / 254
  //   128 caches of ~8,000 rows   206 / 190       351 / 335       122 / 111       184 / 190       269 / 245
  //   4 caches of 24,000          27.3 / 28.7     41.5 / 39.5     18.9 / 22.2     23.5 / 25.4     36.1 / 36.1
  //   one of 12,000               12.9 / 12.7     17.3 / 13.4     9.8 / 9.7       11.1 / 11.3     15.1 / 14.1
  //   one of 30,000               23.6 / 17.6     34.6 / 19.7     15.4 / 12.3     19.8 / 15.3     28.3 / 20.3
  //   4 caches of 8,000           13.6 / 17.3     19.8 / 20.7     10.2 / 14.2     11.7 / 14.8     17.3 / 20.7
  // Lists are all of one length, so clusters are up to 6% better for long ones too, which the rule, made
  // for lengths that it does not know, leaves to stretches.
  int c = 1;
  while (c < kMaxCluster && c * kWarps < steps && s.items * c * 2 <= slots) c *= 2;
  const int most = s.items * c * 4 >= slots ? kMaxShared : kMaxSharedFew;
  if (steps <= int64_t(c) * kWarps * most || s.items >= 64 * slots) {
    s.cluster = c;
    return s;
  }
  s.ctas = int(std::min(slots, (s.items * steps + kMinSteps - 1) / kMinSteps));
  s.bytes = size_t(s.ctas) * 2 * s.hc * (g.D + 4) * 4 + size_t(s.items) * 8;
  return s;
}

template <class T, int BITS, int D, int NC>
cudaError_t launch(const AttnParams& p, const Shape& s, cudaStream_t st) {
  using L = Lay<BITS, D>;
  constexpr int smem = kWarps * L::RING;
  const auto kernel = cache_attn_kernel<T, BITS, D, NC>;
  static std::atomic<uint64_t> set{0};  // devices whose kernel has been given its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(s.ctas ? s.ctas : s.items * s.cluster));
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = unsigned(s.cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = s.cluster > 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess || s.ctas == 0) return e;
  // the join's launch overlaps the kernel's end; few items are spread over more blocks each
  const int64_t wide = std::max<int64_t>(int64_t(sm_count()) * 4 / s.items, 1);
  cfg.gridDim = dim3(unsigned(s.items), unsigned(std::min<int64_t>(wide, s.hc * D / 32)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D>, p, s.hc);
}

template <class T, int BITS, int D>
cudaError_t by_heads(const AttnParams& p, const Shape& s, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (s.hc == 8) return launch<T, BITS, D, 2>(p, s, st);
  return launch<T, BITS, D, 1>(p, s, st);
}

template <class T, int BITS>
cudaError_t by_width(const AttnParams& p, const Shape& s, cudaStream_t st) {
  if (p.c.g.D == 32) return by_heads<T, BITS, 32>(p, s, st);
  if (p.c.g.D == 64) return by_heads<T, BITS, 64>(p, s, st);
  return by_heads<T, BITS, 128>(p, s, st);
}

}  // namespace

size_t cache_fwd_workspace(const CacheParams& p, gattn_dtype dt, int max_keys, bool lists) {
  return shape(p, dt, max_keys, lists).bytes;
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
  p.info = reinterpret_cast<int2*>(p.part + int64_t(s.ctas) * 2 * s.hc * (c.g.D + 4));
  p.groups = s.groups;
  p.ctas = s.ctas;
  p.cluster = s.cluster;
  p.max_keys = max_keys;
  if (s.items * s.cluster > INT32_MAX) {
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
