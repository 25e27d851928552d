// block_select.cu -- the cheap score that chooses blocks: 64-bit sums of
// every block of keys and every unit of queries, scores, and the topk best.
//
// The choice is a whole number that must not hang on the order of a sum, so
// it is defined by scores in 64 bits.  Sums run as pairs of fp32 (each
// addition keeps its exact rounding error in the second member, about 48
// bits, at fp32 rates: this GPU's fp64 units add two numbers a clock and SM,
// a fiftieth of what memory delivers); fp64 appears once per finished sum, and
// for the whole of one that leaves the range of fp32.
// Scores run in fp32 FMAs with an error bound
//   |score - exact| <= e = (D + 32) 2^-23 |q| max|k / n|   (Cauchy-Schwarz),
// a radix select finds the topk-th score T, blocks above T + 2e are in, below
// T - 2e out, and only blocks in between are scored again in fp64.  Where the
// norms leave the range in which that bound holds, all are.  Which blocks the
// causal mask leaves, and which of them come first, follows from positions alone.
//
// Measured: sums over 65,536 nodes of 8 heads of 64 (bf16) 20 us, 3.3 TB/s, with
// issue slots half busy with the exact additions; the choice of 16 of 43 blocks for
// 547 units and 8 heads 21 us, a chain of small phases (scores, radix passes,
// fp64 scores of the undecided) with one to four CTAs an SM; for 8 single tokens
// against caches of about 4,000 keys 4.2 and 11 us.
#include <algorithm>

#include "attn_launch.cuh"
#include "attn_pipe.cuh"
#include "block.cuh"

namespace gattn {

namespace {

constexpr int kThr = 256;

// 16 bytes of a row as fp32
template <class T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int V = 4;
  __device__ static void unpack(uint4 a, float* f) {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int V = 8;
  __device__ static void unpack(uint4 a, float* f) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

struct SumParams {
  BlockGeom g;
  const void* x;
  const int32_t* since;
  double* sums;
  int per, l_heads;  // rows per piece, log2 of the heads of a group
  bool queries;
  int cx;            // 16-byte columns a CTA covers (a power of two)
  int zs;            // since: CTAs that share a sequence's pieces
};

// (a, e) += f, with e the exact rounding errors of a's additions
__device__ __forceinline__ void add_exact(float2& a, float2& e, float2 f) {
  const float2 minus = f2s(-1.f);
  const float2 t = f2add(a, f);
  const float2 b = f2fma(a, minus, t);                     // what f became
  const float2 c = f2fma(f2fma(b, minus, t), minus, a);    // what a lost
  e = f2add(e, f2add(c, f2fma(b, minus, f)));
  a = t;
}

// A CTA sums 16-byte columns [blockIdx.y * cx, + cx) of the Hkv * D sums of
// one piece (or, with `since`, of a sequence's pieces from there on).
// 256 / cx strands share the piece's (row, head) pairs; their (sum, error)
// pairs meet in shared memory in strand order.
template <class T>
__global__ void __launch_bounds__(kThr, 4) piece_sums_kernel(const SumParams p) {
  constexpr int V = Vec16<T>::V;
  __shared__ float2 sh[kThr * V];
  const BlockGeom& g = p.g;
  const int32_t* beg = p.queries ? g.seq_q : g.seq_k;
  const int s = p.since ? blockIdx.x : piece_seq(beg, g.S, p.per, blockIdx.x);
  const Span sp = p.queries ? span_q(g, s) : span_k(g, s);
  const int base = piece_base(beg, s, p.per), rows = p.queries ? g.U : g.B;
  const int cx = p.cx, tx = threadIdx.x & (cx - 1), ty = threadIdx.x / cx, ny = kThr / cx;
  const int W = g.Hkv * g.D, heads = 1 << p.l_heads;
  const int col = (blockIdx.y * cx + tx) * V;  // of Hkv * D
  int j = blockIdx.x - base, step = 1, last = j;  // pieces of the sequence
  if (p.since) {
    j = max(p.since[s], 0) / p.per + blockIdx.z;
    step = p.zs;
    last = (sp.len + p.per - 1) / p.per - 1;
  }
  for (; j <= last; j += step) {
    const int piece = base + j;
    const int64_t pos = int64_t(j) * p.per;
    const int n = pos >= 0 && pos < sp.len ? (int)min(int64_t(p.per), sp.len - pos) : 0;
    if (piece >= rows) break;
    float2 a[V / 2], e[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) a[i] = e[i] = make_float2(0.f, 0.f);
    if (col < W) {
      const int kh = col / g.D, d = col - kh * g.D;
      const T* x = static_cast<const T*>(p.x) + (((sp.beg + pos) * W) << p.l_heads) +
                   int64_t(kh) * heads * g.D + d;
      const int total = n << p.l_heads;
      // four rows are on their way while four are added
      const auto fetch = [&](int i, uint4* to) {
#pragma unroll
        for (int q = 0; q < 4; ++q, i += ny)
          to[q] = i < total ? *reinterpret_cast<const uint4*>(
                                  x + ((int64_t(i >> p.l_heads) * W) << p.l_heads) +
                                  int64_t(i & (heads - 1)) * g.D)
                            : make_uint4(0, 0, 0, 0);
      };
      const auto add = [&](const uint4* from) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float f[V];
          Vec16<T>::unpack(from[q], f);
#pragma unroll
          for (int k = 0; k < V / 2; ++k)
            add_exact(a[k], e[k], make_float2(f[2 * k], f[2 * k + 1]));
        }
      };
      uint4 r0[4], r1[4];
      fetch(ty, r0);
      for (int i = ty; i < total; i += 8 * ny) {
        fetch(i + 4 * ny, r1);
        add(r0);
        if (i + 4 * ny >= total) break;
        fetch(i + 8 * ny, r0);
        add(r1);
      }
    }
    __syncthreads();  // the last piece's sums have been read
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      sh[ty * cx * V + tx * V + 2 * i] = make_float2(a[i].x, e[i].x);
      sh[ty * cx * V + tx * V + 2 * i + 1] = make_float2(a[i].y, e[i].y);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cx * V; c += kThr) {
      float2 t = sh[c];
      for (int y = 1; y < ny; ++y) {
        const float2 f = sh[y * cx * V + c];
        float2 aa = make_float2(t.x, 0.f), ee = make_float2(t.y, 0.f);
        add_exact(aa, ee, make_float2(f.x, 0.f));
        t = make_float2(aa.x, ee.x + f.y);
      }
      const int o = blockIdx.y * cx * V + c;
      if (o >= W) continue;
      double sum = double(t.x) + double(t.y);
      if (!(fabsf(t.x) <= 3.4e38f)) {  // beyond fp32, on the way at least: again in fp64
        const int kh = o / g.D, d = o - kh * g.D;
        const T* x = static_cast<const T*>(p.x) + (((sp.beg + pos) * W) << p.l_heads) +
                     int64_t(kh) * heads * g.D + d;
        sum = 0.0;
        for (int i = 0; i < n << p.l_heads; ++i)
          sum += double(float(x[((int64_t(i >> p.l_heads) * W) << p.l_heads) +
                                int64_t(i & (heads - 1)) * g.D]));
      }
      p.sums[int64_t(piece) * W + o] = sum;
    }
  }
}

// --------------------------------------------------------------------------
// scores and the topk best
// --------------------------------------------------------------------------
struct SelParams {
  BlockGeom g;
  const void* Q;         // used when units are single rows
  const double* qsum;    // [U][Hkv][D] else
  const double* sums;    // [B][Hkv][D]
  int32_t* idx;
  int cap;               // blocks of a sequence that are looked at
};

// fp64 to fp32, rounded towards zero, with integer instructions (the
// conversion instruction runs at the fp64 rate).
__device__ __forceinline__ float trunc32(double x) {
  const uint32_t hi = __double2hiint(x), lo = __double2loint(x);
  const uint32_t ex = (hi >> 20) & 0x7ff;
  uint32_t m = (__funnelshift_l(lo, hi, 3) - (896u << 23)) & 0x7fffffffu;
  m = ex <= 896 ? 0u : ex >= 1151 ? 0x7f800000u : m;
  if (ex == 0x7ff && ((hi & 0xfffff) | lo)) m = 0x7fc00000u;
  return __uint_as_float(m | (hi & 0x80000000u));
}

__device__ __forceinline__ uint32_t order_key(float x) {  // larger score, larger key (finite x)
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are one score
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The k-th largest of n keys (1 <= k <= n), by one warp; hist: 256 words.
__device__ uint32_t kth_key(const double* sc, int n, int k, uint32_t* hist) {
  const int lane = threadIdx.x & 31;
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hist[lane * 8 + i] = 0;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
      const uint32_t key = order_key(reinterpret_cast<const float*>(sc + i)[0]);
      if ((key & mask) == prefix) atomicAdd(hist + ((key >> shift) & 255), 1u);
    }
    __syncwarp();
    uint32_t mine = 0;  // lane l: bins [8 l, 8 l + 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += hist[lane * 8 + i];
    uint32_t above = mine;  // suffix sum over lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_down_sync(0xffffffffu, above, o);
      if (lane + o < 32) above += t;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, above >= uint32_t(k));
    const int who = 31 - __clz(reach);  // highest lane whose suffix holds k keys
    uint32_t bin = 0, left = 0;
    if (lane == who) {
      uint32_t c = above - mine;
      int b = 7;
      for (; b > 0 && c + hist[lane * 8 + b] < uint32_t(k); --b) c += hist[lane * 8 + b];
      bin = lane * 8 + b;
      left = k - c;
    }
    bin = __shfl_sync(0xffffffffu, bin, who);
    k = __shfl_sync(0xffffffffu, left, who);
    prefix |= bin << shift;
    mask |= 255u << shift;
    __syncwarp();
  }
  return prefix;
}

// UT consecutive units of one key head per CTA.  A score entry is 8 bytes:
// the fp32 score, or the fp64 score of a block near the last place.
template <class T, int UT>
__global__ void __launch_bounds__(kThr, 4) select_kernel(const SelParams p) {
  extern __shared__ __align__(16) double sm[];
  const BlockGeom& g = p.g;
  const int D = g.D, kh = blockIdx.y;
  double* q64 = sm;                                        // [UT][D]
  float* q32 = reinterpret_cast<float*>(q64 + UT * D);     // [UT][D]
  uint32_t* hist = reinterpret_cast<uint32_t*>(q32 + UT * D);  // [UT][256]
  double* sc = reinterpret_cast<double*>(hist + UT * 256);     // [UT][cap]
  __shared__ float wmax[kThr / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u0 = blockIdx.x * UT, u1 = min(u0 + UT, g.U);

  for (int ub = u0; ub < u1;) {
    // the units from ub on that belong to ub's sequence
    const Unit un = unit_at(g, ub);
    const int end = un.s + 1 < g.S ? piece_base(g.seq_q, un.s + 1, g.qb) : g.U;
    const int cnt = max(1, min(u1, end) - ub);
    const Span qs = span_q(g, un.s), ks = span_k(g, un.s);
    const int b0 = piece_base(g.seq_k, un.s, g.block);
    const int nb = max(0, min(min((ks.len + g.block - 1) / g.block, p.cap), g.B - b0));
    const int first_unit = piece_base(g.seq_q, un.s, g.qb);
    __syncthreads();
    for (int i = threadIdx.x; i < UT * D; i += kThr) {
      const int j = i / D, d = i - j * D, u = ub + j;
      double v = 0.0;
      const int64_t off = int64_t(u - first_unit) * g.qb;
      if (j < cnt && off >= 0 && off < qs.len) {
        if (p.qsum) {
          v = p.qsum[(int64_t(u) * g.Hkv + kh) * D + d];
        } else {
          const T* q = static_cast<const T*>(p.Q) + ((qs.beg + off) * g.H + kh * g.G) * D + d;
          for (int h = 0; h < g.G; ++h) v += double(float(q[h * D]));
        }
      }
      q64[i] = v;
      q32[i] = trunc32(v);
    }
    __syncthreads();

    // scores: 8 lanes per block, each D / 8 of its columns (pairs)
    float big = 0.f;  // largest |k|^2 / n^2
    const int sub = threadIdx.x & 7;
    for (int b = threadIdx.x >> 3; b < ((nb + 31) & ~31); b += kThr / 8) {
      float acc[UT];
#pragma unroll
      for (int j = 0; j < UT; ++j) acc[j] = 0.f;
      float nn = 0.f;
      const bool in = b < nb;
      const double* k = p.sums + (int64_t(b0 + (in ? b : 0)) * g.Hkv + kh) * D;
      if (in) {
        if (D >= 16) {
#pragma unroll 4
          for (int d = sub * 2; d < D; d += 16) {
            const double2 kk = *reinterpret_cast<const double2*>(k + d);
            const float x = trunc32(kk.x), y = trunc32(kk.y);
            nn = fmaf(x, x, fmaf(y, y, nn));
#pragma unroll
            for (int j = 0; j < UT; ++j) {
              const float2 q = *reinterpret_cast<const float2*>(q32 + j * D + d);
              acc[j] = fmaf(x, q.x, fmaf(y, q.y, acc[j]));
            }
          }
        } else if (sub < D) {
          const float x = trunc32(k[sub]);
          nn = x * x;
#pragma unroll
          for (int j = 0; j < UT; ++j) acc[j] = x * q32[j * D + sub];
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        nn += __shfl_xor_sync(0xffffffffu, nn, o);
#pragma unroll
        for (int j = 0; j < UT; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      }
      if (in) {
        const float inv = 1.f / float(min(g.block, ks.len - b * g.block));
        big = fmaxf(big, nn * inv * inv);
        if (nn != nn) big = __int_as_float(0x7f800000);
        if (sub == 0)
#pragma unroll
          for (int j = 0; j < UT; ++j)
            reinterpret_cast<float*>(sc + j * p.cap + b)[0] = acc[j] * inv;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) wmax[warp] = big;
    __syncthreads();

    // one warp per unit
    for (int j = warp; j < cnt; j += kThr / 32) {
      double* s = sc + j * p.cap;
      int32_t* out = p.idx + (int64_t(ub + j) * g.Hkv + kh) * g.topk;
      // blocks [0, far) compete; [far, end) reach the unit's own positions and come first
      const int64_t off = int64_t(ub + j - first_unit) * g.qb;
      int end = off >= 0 && off < qs.len ? nb : 0, far = end;
      if (g.causal && end > 0) {
        const int64_t first = off + ks.len - qs.len;
        const int64_t last = min(off + g.qb, int64_t(qs.len)) + ks.len - qs.len - 1;
        end = last < 0 ? 0 : int(min(int64_t(end), last / g.block + 1));
        far = first < 0 ? 0 : int(min(int64_t(end), first / g.block));
      }
      end = min(end, far + g.topk);
      const int k = min(g.topk - (end - far), far);  // of those that compete
      float qn = 0.f, kn = 0.f;  // |q|^2, largest |k|^2 / n^2
      for (int d = lane; d < D; d += 32) qn = fmaf(q32[j * D + d], q32[j * D + d], qn);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) qn += __shfl_xor_sync(0xffffffffu, qn, o);
#pragma unroll
      for (int w = 0; w < kThr / 32; ++w) kn = fmaxf(kn, wmax[w]);
      // Between these norms nothing overflows (a score's sum stays below 2^123) and what
      // underflows (values below 2^-126, that times the other norm) is far below the bound.
      // Otherwise -- among them norms of 0, infinite or not a number -- the fp32 scores
      // say nothing and all that compete are scored in fp64.
      constexpr float kLeast = 0x1p-116f, kMost = 0x1p116f;
      const bool sound = qn >= kLeast && qn <= kMost && kn >= kLeast && kn <= kMost;
      float lo = neg_inf(), hi = -neg_inf();  // below lo: out; above hi: in; between: by fp64
      bool exact = k > 0 && !sound;
      int need = k;
      if (sound && k > 0 && far > k) {
        const float kth = key_score(kth_key(s, far, k, hist + j * 256));
        const float e = float(D + 32) * 0x1p-23f * sqrtf(qn) * sqrtf(kn) * 1.0001f;
        lo = kth - 2.f * e;
        hi = kth + 2.f * e;
        // count the sure ones; when those between are exactly what is missing, take them all
        int sure = 0, mid = 0;
        for (int i = lane; i < far; i += 32) {
          const float v = reinterpret_cast<const float*>(s + i)[0];
          sure += v > hi;
          mid += v >= lo && v <= hi;
        }
        need = k - __reduce_add_sync(0xffffffffu, sure);
        exact = __reduce_add_sync(0xffffffffu, mid) > need;
      }
      constexpr long long kOut = 0x7ff8000000000001LL, kIn = 0x7ff8000000000002LL;
      if (exact) {
        // score those between in fp64: one block at a time, the lanes over D
        for (int i0 = 0; i0 < far; i0 += 32) {
          const int i = i0 + lane;
          const float v = i < far ? reinterpret_cast<const float*>(s + i)[0] : 0.f;
          unsigned todo =
              __ballot_sync(0xffffffffu, i < far && (!sound || (v >= lo && v <= hi)));
          long long mine = sound && v > hi ? kIn : kOut;
          while (todo) {
            const int l = __ffs(todo) - 1;
            todo &= todo - 1;
            const int b = i0 + l;
            const double* kk = p.sums + (int64_t(b0 + b) * g.Hkv + kh) * D;
            double t = 0.0;
            for (int d = lane; d < D; d += 32) t = fma(q64[j * D + d], kk[d], t);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            t /= double(min(g.block, ks.len - b * g.block));
            // (not a number and -inf are never chosen)
            if (lane == l) mine = t > -1.0 / 0.0 ? __double_as_longlong(t) : kOut;
          }
          // the fp64 score of a scored block; others as quiet tags
          if (i < far) s[i] = __longlong_as_double(mine);
        }
        __syncwarp();
        // the `need` best by (score, lower id): take the maximum `need` times
        for (; need > 0; --need) {
          double best = -1.0 / 0.0;
          int at = INT32_MAX;
          for (int i = lane; i < far; i += 32) {
            const double v = s[i];
            if (v == v && (at == INT32_MAX || v > best)) {
              best = v;
              at = i;
            }
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(0xffffffffu, best, o);
            const int oa = __shfl_xor_sync(0xffffffffu, at, o);
            if (oa != INT32_MAX && (at == INT32_MAX || ob > best || (ob == best && oa < at))) {
              best = ob;
              at = oa;
            }
          }
          if (at == INT32_MAX) break;
          __syncwarp();
          if (lane == 0) s[at] = __longlong_as_double(kIn);
          __syncwarp();
        }
      }
      int n = 0;
      for (int i0 = 0; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        bool in = i < end;
        if (i < far)
          in = exact ? __double_as_longlong(s[i]) == kIn
                     : k > 0 && reinterpret_cast<const float*>(s + i)[0] >= lo;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (in) out[n + __popc(m & ((1u << lane) - 1))] = i;
        n += __popc(m);
      }
      for (int i = n + lane; i < g.topk; i += 32) out[i] = -1;
    }
    ub += cnt;
  }
}

gattn_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s launch failed: %s", what, cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  return GATTN_OK;
}

size_t select_smem(int UT, int D, int cap) {
  return size_t(UT) * (D * 12 + 1024 + size_t(cap) * 8);
}

}  // namespace

gattn_status launch_block_sums(const BlockGeom& g, gattn_dtype dt, const void* x, bool queries,
                               const int32_t* since, double* sums, cudaStream_t st) {
  SumParams p{};
  p.g = g;
  p.x = x;
  p.since = since;
  p.sums = sums;
  p.queries = queries;
  p.per = queries ? g.qb : g.block;
  p.l_heads = queries ? 31 - __builtin_clz(g.G) : 0;
  const int V = dt == GATTN_F32 ? 4 : 8;
  const int cols = g.Hkv * g.D / V;  // a power of two
  // 1 KB of a row per CTA; a token's few blocks are read by twice the strands instead
  // (8 sequences, one token: 5.0 -> 4.0 us; all of 65,536 nodes: 19.5 -> 22.6 us)
  p.cx = std::min(cols, since ? 32 : 64);
  const int pieces = queries ? g.U : g.B;
  if (pieces <= 0) return GATTN_OK;
  // from a position on, a sequence has few pieces to renew (one new token: one):
  // CTAs by sequence instead of one that looks and leaves per piece
  p.zs = 4;
  const unsigned ny = unsigned((cols + p.cx - 1) / p.cx);
  const dim3 grid = since ? dim3(g.S, ny, p.zs) : dim3(pieces, ny);
  if (dt == GATTN_F32) piece_sums_kernel<float><<<grid, kThr, 0, st>>>(p);
  else piece_sums_kernel<__nv_bfloat16><<<grid, kThr, 0, st>>>(p);
  return launched("gattn_block_sums");
}

gattn_status launch_block_select(const BlockGeom& g, gattn_dtype dt, const void* Q,
                                 const double* qsum, const double* sums, int max_blocks,
                                 int32_t* idx, cudaStream_t st) {
  SelParams p{};
  p.g = g;
  p.Q = Q;
  p.qsum = qsum;
  p.sums = sums;
  p.idx = idx;
  p.cap = std::max(1, max_blocks);
  // eight units share a pass over the sums where that leaves every SM work;
  // single units otherwise (few units, or more blocks than fit eight times)
  const int sms = sm_count();
  const bool eight = int64_t(g.U) * g.Hkv >= int64_t(16) * sms &&
                     select_smem(8, g.D, p.cap) <= size_t(200) * 1024;
  const int UT = eight ? 8 : 1;
  const size_t bytes = select_smem(UT, g.D, p.cap);
  if (bytes > size_t(220) * 1024) {
    set_error("gattn_block_select: %d blocks in a sequence are too many (at most %d)", p.cap,
              int((220 * 1024 - g.D * 12 - 1024) / 8));
    return GATTN_ERR_UNSUPPORTED;
  }
  const dim3 grid((g.U + UT - 1) / UT, g.Hkv);
  auto go = [&](auto kern) -> gattn_status {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e != cudaSuccess) {
      set_error("gattn_block_select: %s", cudaGetErrorString(e));
      return GATTN_ERR_CUDA;
    }
    kern<<<grid, kThr, bytes, st>>>(p);
    return launched("gattn_block_select");
  };
  if (dt == GATTN_F32) return eight ? go(select_kernel<float, 8>) : go(select_kernel<float, 1>);
  return eight ? go(select_kernel<__nv_bfloat16, 8>) : go(select_kernel<__nv_bfloat16, 1>);
}

}  // namespace gattn
