// block_simt.cu -- block attention on the CUDA cores, for fp32 tensors (the
// tensor cores' kinds keep fewer than 24 bits of a product's operands).
//
// 64 x 64 score tiles: 256 threads hold 4 x 4 scores each, operands are staged
// in shared memory by cp.async (four threads a row), and a thread's 4 rows of
// the output (or gradient) stay in registers.  A step of 64 rows by 64 keys is
// 2 (forward), 3 (dQ) or 4 (dK, dV) products of 64 x 64 x D on the FMA units; up
// to D = 64 the next step's operands are fetched meanwhile.  At D <= 32 a row
// of the last products has 8 float4, so the other 8 threads of the 16 take every
// second group of four keys.
//
// With the unit's block list ascending, the keys a row may see are the first
// columns of its steps, so the mask of a row is one number (list_keys).
//
// Measured: 7 graphs of 429 nodes, 4 heads of 32, 8 blocks of 32: forward 25 us,
// dQ 32 us, dK and dV 63 us (1.4 GFLOP together, in half-empty rounds of the 304
// CTAs that are resident).
#include <algorithm>

#include "attn_launch.cuh"
#include "block.cuh"

namespace gattn {

namespace {

constexpr int kR = 64;     // rows of a tile
constexpr int kC = 64;     // keys of a step
constexpr int kThr = 256;
constexpr int kPS = kC + 4;  // row stride of the score tile

// Operand buffers of a step, and CTAs of an SM: two up to D = 64, where shared
// memory and registers allow them.
template <int DQ>
constexpr int kBufs = DQ < 2 ? 2 : 1;

struct FwdP {
  BlockGeom g;
  const float *Q, *K, *V;
  const int32_t* idx;
  float* out;
  float* lse;
};

// element offset of the (row, head) pair r of a unit, -1 past its rows
__device__ __forceinline__ int64_t q_off(const BlockGeom& g, const Unit& u, int kh, int r) {
  const int t = r / g.G;
  if (t >= u.n) return -1;
  return (int64_t(u.row + t) * g.H + kh * g.G + (r - t * g.G)) * g.D;
}

// 64 rows of D elements to shared memory (row stride D + 4), asynchronously;
// off(r) < 0: zeros.  Returns the offset of this thread's row, threadIdx.x / 4.
template <class F>
__device__ __forceinline__ int64_t stage(float* dst, const float* src, int D, F off) {
  const int r = threadIdx.x >> 2;
  const int64_t o = off(r);
  const float* s = src + (o >= 0 ? o : 0);
  const uint32_t d0 = smem_u32(dst + r * (D + 4)), bytes = o >= 0 ? 16 : 0;
  for (int d = (threadIdx.x & 3) * 4; d < D; d += 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d0 + d * 4), "l"(s + d),
                 "r"(bytes)
                 : "memory");
  return o;
}
// Closes the group of the copies so far.  landed() waits for closed groups alone, so
// every path from a stage() to a landed() passes one, those that take no step too.
__device__ __forceinline__ void staged() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void landed() {  // all groups but the last N
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
  __syncthreads();
}

// s[i][j] = a[4 ty + i] . b[tx + 16 j]
__device__ __forceinline__ void dots(const float* a, const float* b, int D, float s[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ld = D + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * 4 + i) * ld + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ld + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z,
                  fmaf(x[i].w, y[j].w, s[i][j]))));
  }
}

// o[i][*] += sum_k w(4 ty + i, k) b[k][cols of this thread], cols 4 tx + 64 q;
// DQ = 0 (D <= 32): cols 4 (tx % 8), of every second four k.
// TR: w is stored [k][row].  GUARD: a zero weight takes nothing from its row
// of b, which may hold non-finite values that the row must not see.
template <int DQ, bool TR, bool GUARD>
__device__ __forceinline__ void weighted(const float* w, const float* b, int D, float (*o)[4]) {
  constexpr int N = DQ ? DQ : 1;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ld = D + 4;
  const int c0 = (DQ ? tx : tx & 7) * 4;
#pragma unroll 2
  for (int k = DQ ? 0 : (tx >> 3) * 4; k < kC; k += DQ ? 4 : 8) {
    float x[4][4];  // [key][row]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(TR ? w + (k + i) * kPS + ty * 4
                                                           : w + (ty * 4 + i) * kPS + k);
      if (TR) {
        x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
      } else {
        x[0][i] = v.x; x[1][i] = v.y; x[2][i] = v.z; x[3][i] = v.w;
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int c = c0 + 64 * q;
      if (c >= D) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(b + (k + e) * ld + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (GUARD && x[e][i] == 0.f) continue;
          float* y = o[i * N + q];
          y[0] = fmaf(x[e][i], v.x, y[0]);
          y[1] = fmaf(x[e][i], v.y, y[1]);
          y[2] = fmaf(x[e][i], v.z, y[2]);
          y[3] = fmaf(x[e][i], v.w, y[3]);
        }
      }
    }
  }
}

// row i's columns of this thread, all keys together, times mul: put(column, values)
template <int DQ, class F>
__device__ __forceinline__ void finish(float (*o)[4], int i, int D, float mul, F put) {
  constexpr int N = DQ ? DQ : 1;
  const int tx = threadIdx.x & 15;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    float* y = o[i * N + q];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!DQ) y[e] += __shfl_xor_sync(0xffffffffu, y[e], 8);
      y[e] *= mul;
    }
    const int c = (DQ ? tx : tx & 7) * 4 + 64 * q;
    if (c < D && (DQ || tx < 8)) put(c, make_float4(y[0], y[1], y[2], y[3]));
  }
}

// key row (element offset of K, V) of column c of the step that starts at
// list key k0, -1 past the list
__device__ __forceinline__ int64_t k_off(const BlockGeom& g, const int* ids, int total, int k0,
                                         int c, int kbeg, int kh) {
  const int k = k0 + c;
  if (k >= total) return -1;
  return (int64_t(kbeg + ids[k / g.block] * g.block + k % g.block) * g.Hkv + kh) * g.D;
}

template <int DQ>
__global__ void __launch_bounds__(kThr, kBufs<DQ>) block_fwd_simt(const FwdP p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int ids[kBlkMaxTopk];
  __shared__ int n_ids;
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4, kh = blockIdx.y, u = blockIdx.x, r0 = blockIdx.z * kR;
  constexpr int NB = kBufs<DQ>, N = DQ ? DQ : 1;
  float *sQ = sm, *sK = sQ + kR * ld, *sV = sK + NB * kC * ld, *sP = sV + NB * kC * ld;
  const Unit un = unit_at(g, u);
  if (r0 >= un.n * g.G) return;
  const Span ks = span_k(g, un.s);
  if (threadIdx.x < 32) {
    const int n = block_list(p.idx + u * g.is_u + kh * g.is_h, g.topk,
                             (ks.len + g.block - 1) / g.block, ids);
    if (threadIdx.x == 0) n_ids = n;
  }
  __syncthreads();
  const int n = n_ids, total = list_keys(ids, n, g.block, ks.len);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int lim[4];
  int lim0 = total;  // keys every row of the tile sees
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (r0 + ty * 4 + i) / g.G;
    lim[i] = !g.causal ? total : list_keys(ids, n, g.block, min(un.pos + t + 1, ks.len));
    if (t >= un.n) lim[i] = 0;
  }
  if (g.causal) lim0 = list_keys(ids, n, g.block, min(un.pos + r0 / g.G + 1, ks.len));
  const auto fetch = [&](int k0, int buf) {
    const auto off = [&](int c) { return k_off(g, ids, total, k0, c, ks.beg, kh); };
    stage(sK + buf * kC * ld, p.K, D, off);
    stage(sV + buf * kC * ld, p.V, D, off);
    staged();
  };
  stage(sQ, p.Q, D, [&](int r) { return q_off(g, un, kh, r0 + r); });
  staged();
  if (NB == 2) fetch(0, 0);
  float m[4], l[4], o[4 * N][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = neg_inf();
    l[i] = 0.f;
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i * N + q][e] = 0.f;
  }
  for (int k0 = 0, buf = 0; k0 < total; k0 += kC, buf = NB - 1 - buf) {
    if (k0) __syncthreads();  // the buffer has been read
    if (NB == 1 || k0 + kC < total) fetch(NB == 2 ? k0 + kC : k0, NB - 1 - buf);
    else staged();  // (an empty group)
    landed<NB - 1>();
    float s[4][4];
    dots(sQ, sK + buf * kC * ld, D, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = k0 + tx + 16 * j < lim[i] ? s[i][j] * g.qmul : neg_inf();
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float base = mx == neg_inf() ? 0.f : mx;
      const float corr = ex2(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = ex2(s[i][j] - base);
        sP[(ty * 4 + i) * kPS + tx + 16 * j] = w;
        sum += w;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * corr + sum;
      m[i] = mx;
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i * N + q][e] *= corr;
    }
    __syncwarp();  // a row's weights come from the half-warp that uses them
    if (k0 + kC > lim0) weighted<DQ, false, true>(sP, sV + buf * kC * ld, D, o);
    else weighted<DQ, false, false>(sP, sV + buf * kC * ld, D, o);
  }
  landed<0>();  // with an empty list nothing has waited for Q
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = q_off(g, un, kh, r0 + ty * 4 + i);
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    if (tx == 0 && at >= 0) p.lse[at / D] = l[i] != 0.f ? (m[i] + lg2(l[i])) * kLn2 : neg_inf();
    finish<DQ>(o, i, D, inv, [&](int c, float4 v) {
      if (at >= 0) *reinterpret_cast<float4*>(p.out + at + c) = v;
    });
  }
}

// dQ of 64 (row, head) pairs of a unit
template <int DQ>
__global__ void __launch_bounds__(kThr, kBufs<DQ>) block_dq_simt(const BlockBwdParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int ids[kBlkMaxTopk];
  __shared__ int n_ids;
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4, kh = blockIdx.y, u = blockIdx.x, r0 = blockIdx.z * kR;
  constexpr int NB = kBufs<DQ>, N = DQ ? DQ : 1;
  float *sQ = sm, *sO = sQ + kR * ld, *sK = sO + kR * ld, *sV = sK + NB * kC * ld,
        *sP = sV + NB * kC * ld;
  const Unit un = unit_at(g, u);
  if (r0 >= un.n * g.G) return;
  const Span ks = span_k(g, un.s);
  if (threadIdx.x < 32) {
    const int n = block_list(p.idx + u * g.is_u + kh * g.is_h, g.topk,
                             (ks.len + g.block - 1) / g.block, ids);
    if (threadIdx.x == 0) n_ids = n;
  }
  __syncthreads();
  const int n = n_ids, total = list_keys(ids, n, g.block, ks.len);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int lim[4];
  float L[4], Dl[4], o[4 * N][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i, t = r / g.G;
    lim[i] = !g.causal ? total : list_keys(ids, n, g.block, min(un.pos + t + 1, ks.len));
    if (t >= un.n) lim[i] = 0;
    const int64_t at = q_off(g, un, kh, r);
    const float2 stat = at >= 0 ? p.stat[at / D] : make_float2(0.f, 0.f);
    L[i] = stat.x;
    Dl[i] = stat.y;
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i * N + q][e] = 0.f;
  }
  const auto fetch = [&](int k0, int buf) {
    const auto off = [&](int c) { return k_off(g, ids, total, k0, c, ks.beg, kh); };
    stage(sK + buf * kC * ld, static_cast<const float*>(p.K), D, off);
    stage(sV + buf * kC * ld, static_cast<const float*>(p.V), D, off);
    staged();
  };
  const auto qo = [&](int r) { return q_off(g, un, kh, r0 + r); };
  stage(sQ, static_cast<const float*>(p.Q), D, qo);
  stage(sO, static_cast<const float*>(p.dO), D, qo);
  staged();
  if (NB == 2) fetch(0, 0);
  for (int k0 = 0, buf = 0; k0 < total; k0 += kC, buf = NB - 1 - buf) {
    if (k0) __syncthreads();  // the buffer has been read
    if (NB == 1 || k0 + kC < total) fetch(NB == 2 ? k0 + kC : k0, NB - 1 - buf);
    else staged();  // (an empty group)
    landed<NB - 1>();
    float s[4][4], dp[4][4];
    dots(sQ, sK + buf * kC * ld, D, s);
    dots(sO, sV + buf * kC * ld, D, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = k0 + tx + 16 * j < lim[i];
        const float w = in ? ex2(fmaf(s[i][j], g.qmul, -L[i])) * (dp[i][j] - Dl[i]) : 0.f;
        sP[(ty * 4 + i) * kPS + tx + 16 * j] = w;
      }
    __syncwarp();
    weighted<DQ, false, false>(sP, sK + buf * kC * ld, D, o);
  }
  landed<0>();  // with an empty list nothing has waited for Q and dO
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = q_off(g, un, kh, r0 + ty * 4 + i);
    finish<DQ>(o, i, D, g.scale, [&](int c, float4 v) {
      if (at >= 0) *reinterpret_cast<float4*>(static_cast<float*>(p.dQ) + at + c) = v;
    });
  }
}

// dK, dV of one half (64 keys) of a work item's key tile
template <int DQ>
__global__ void __launch_bounds__(kThr, kBufs<DQ>) block_dkv_simt(const BlockBwdParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int list[1024];
  __shared__ uint8_t mask[1024];
  __shared__ int n_list, n_all;
  constexpr int NB = kBufs<DQ>, N = DQ ? DQ : 1;
  __shared__ float2 row_stat[NB][kR];  // of a step's rows: (lse log2e, Delta),
  __shared__ int row_end[NB][kR];      // the first position that the row does not see
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4;
  float *sK = sm, *sV = sK + kC * ld, *sQ = sV + kC * ld, *sO = sQ + NB * kR * ld,
        *sP = sO + NB * kR * ld;
  float* sS = sP + kR * kPS;
  const int parts = (g.qb * g.G + kR - 1) / kR;  // steps of a unit
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t n_items = p.head[0];
  for (int64_t it = blockIdx.x; it < 2 * n_items; it += gridDim.x) {
    const int4 q = p.items[it >> 1];
    const int half = int(it & 1), kt = q.x / g.Hkv, kh = q.x - kt * g.Hkv;
    const int s = piece_seq(g.seq_k, g.S, kBlkTile, kt);
    const Span ks = span_k(g, s), qs = span_q(g, s);
    const int tpos = (kt - piece_base(g.seq_k, s, kBlkTile)) * kBlkTile;
    const int pos0 = tpos + half * kC;
    if (pos0 >= ks.len) continue;
    const int bl0 = tpos / g.block, per = kBlkTile / g.block;
    const int nb = min(per, (ks.len + g.block - 1) / g.block - bl0);
    const int brow = min(piece_base(g.seq_k, s, g.block) + bl0, g.B - nb);
    const int ub = piece_base(g.seq_q, s, g.qb), nu = (qs.len + g.qb - 1) / g.qb;
    const auto ko = [&](int c) -> int64_t {
      return pos0 + c < ks.len ? (int64_t(ks.beg + pos0 + c) * g.Hkv + kh) * D : -1;
    };
    __syncthreads();
    stage(sK, static_cast<const float*>(p.K), D, ko);
    stage(sV, static_cast<const float*>(p.V), D, ko);
    staged();
    int blk[4];  // block of this thread's keys within the tile
#pragma unroll
    for (int j = 0; j < 4; ++j) blk[j] = (half * kC + tx + 16 * j) / g.block;
    float gk[4 * N][4], gv[4 * N][4];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) gk[i][e] = gv[i][e] = 0.f;
    int seen = 0;  // units of the key tile before this group of bitmap words
    for (int w0 = ub / 32; w0 <= (ub + nu - 1) / 32 && nu > 0 && seen < q.y + q.z; w0 += 32) {
      __syncthreads();
      if (threadIdx.x < 32) {  // the units of 32 words that belong to the item
        const int w = w0 + threadIdx.x;
        uint32_t bits[8], any = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          bits[b] = b < nb && w < p.words
                        ? p.bits[(int64_t(brow + b) * g.Hkv + kh) * p.words + w] : 0u;
          any |= bits[b];
        }
        const int c = __popc(any);
        int before = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, before, o);
          if (threadIdx.x >= o) before += t;
        }
        const int all = __shfl_sync(0xffffffffu, before, 31);
        int at = seen + before - c;
        for (uint32_t a = any; a; a &= a - 1, ++at) {
          if (at < q.y || at >= q.y + q.z) continue;
          const int bit = __ffs(a) - 1;
          uint32_t mk = 0;
#pragma unroll
          for (int b = 0; b < 8; ++b) mk |= ((bits[b] >> bit) & 1u) << b;
          const int i = at - max(seen, q.y);
          list[i] = w * 32 + bit;
          mask[i] = uint8_t(mk);
        }
        if (threadIdx.x == 0) {
          n_list = max(0, min(seen + all, q.y + q.z) - max(seen, q.y));
          n_all = all;
        }
      }
      __syncthreads();
      const int nl = n_list;
      seen += n_all;
      const int steps = nl * parts;
      const auto fetch = [&](int st, int buf) {
        const int e = st / parts, r0 = (st - e * parts) * kR;
        const int64_t uo = int64_t(list[e] - ub) * g.qb;
        Unit un{};
        un.s = s;
        // (a unit outside the sequence: only where offsets lie about the tables)
        if (uo >= 0 && uo < qs.len) {
          un.row = qs.beg + int(uo);
          un.n = min(g.qb, qs.len - int(uo));
          un.pos = int(uo) + ks.len - qs.len;
        }
        const auto qo = [&](int r) { return q_off(g, un, kh, r0 + r); };
        const int64_t at = stage(sQ + buf * kR * ld, static_cast<const float*>(p.Q), D, qo);
        stage(sO + buf * kR * ld, static_cast<const float*>(p.dO), D, qo);
        staged();
        if ((threadIdx.x & 3) == 0) {
          const int r = threadIdx.x >> 2;
          row_stat[buf][r] = at >= 0 ? p.stat[at / D] : make_float2(0.f, 0.f);
          row_end[buf][r] =
              at < 0 ? 0 : g.causal ? min(un.pos + (r0 + r) / g.G + 1, ks.len) : ks.len;
        }
      };
      if (NB == 2 && steps) fetch(0, 0);
      for (int st = 0, buf = 0; st < steps; ++st, buf = NB - 1 - buf) {
        const uint32_t mk = mask[st / parts];
        if (st) __syncthreads();  // the buffer has been read
        if (NB == 1 || st + 1 < steps) fetch(NB == 2 ? st + 1 : st, NB - 1 - buf);
        else staged();  // (an empty group)
        landed<NB - 1>();
        float sc[4][4], dp[4][4];
        dots(sQ + buf * kR * ld, sK, D, sc);
        dots(sO + buf * kR * ld, sV, D, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 stat = row_stat[buf][ty * 4 + i];
          const int end = row_end[buf][ty * 4 + i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const bool in = pos0 + c < end && ((mk >> blk[j]) & 1u);
            const float w = in ? ex2(fmaf(sc[i][j], g.qmul, -stat.x)) : 0.f;
            sP[(ty * 4 + i) * kPS + c] = w;
            sS[(ty * 4 + i) * kPS + c] = in ? w * (dp[i][j] - stat.y) : 0.f;
          }
        }
        __syncthreads();
        weighted<DQ, true, false>(sP, sO + buf * kR * ld, D, gv);
        weighted<DQ, true, false>(sS, sQ + buf * kR * ld, D, gk);
      }
    }
    landed<0>();  // an item without units has not waited for K and V, which the next overwrites
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = ty * 4 + i;
      const int64_t at = ko(c);
      float* part = p.part + (int64_t(max(q.w, 0)) * 2 * kBlkTile + half * kC + c) * D;
      finish<DQ>(gk, i, D, q.w < 0 ? g.scale : 1.f, [&](int d, float4 v) {
        if (at >= 0)
          *reinterpret_cast<float4*>((q.w < 0 ? static_cast<float*>(p.dK) + at : part) + d) = v;
      });
      part += int64_t(kBlkTile) * D;
      finish<DQ>(gv, i, D, 1.f, [&](int d, float4 v) {
        if (at >= 0)
          *reinterpret_cast<float4*>((q.w < 0 ? static_cast<float*>(p.dV) + at : part) + d) = v;
      });
    }
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

template <class K, class P>
gattn_status go(K kern, dim3 grid, int floats, const P& p, cudaStream_t st, const char* what) {
  const int bytes = floats * 4;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) {
    set_error("%s: %s", what, cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  kern<<<grid, kThr, bytes, st>>>(p);
  return launched(what);
}

dim3 row_grid(const BlockGeom& g) {
  return dim3(unsigned(g.U), unsigned(g.Hkv), unsigned((g.qb * g.G + kR - 1) / kR));
}

}  // namespace

gattn_status launch_block_fwd_simt(const BlockGeom& g, const float* Q, const float* K,
                                   const float* V, const int32_t* idx, float* out, float* lse,
                                   cudaStream_t st) {
  const FwdP p{g, Q, K, V, idx, out, lse};
  const auto run = [&](auto kern, int bufs) {
    return go(kern, row_grid(g), (1 + 2 * bufs) * kR * (g.D + 4) + kR * kPS, p, st,
              "gattn_block_fwd");
  };
  return g.D <= 32   ? run(block_fwd_simt<0>, kBufs<0>)
         : g.D <= 64 ? run(block_fwd_simt<1>, kBufs<1>)
                     : run(block_fwd_simt<2>, kBufs<2>);
}

gattn_status launch_block_bwd_simt(const BlockBwdParams& p, cudaStream_t st) {
  const BlockGeom& g = p.g;
  const int tile = kR * (g.D + 4);
  const auto dq = [&](auto kern, int bufs) {
    return go(kern, row_grid(g), (2 + 2 * bufs) * tile + kR * kPS, p, st, "gattn_block_bwd (dQ)");
  };
  const dim3 gk(unsigned(std::min<int64_t>(2 * p.max_items, int64_t(sm_count()) * 2)));
  const auto dkv = [&](auto kern, int bufs) {
    return go(kern, gk, (2 + 2 * bufs) * tile + 2 * kR * kPS, p, st, "gattn_block_bwd (dK, dV)");
  };
  gattn_status s = GATTN_OK;
  if (g.U > 0)
    s = g.D <= 32   ? dq(block_dq_simt<0>, kBufs<0>)
        : g.D <= 64 ? dq(block_dq_simt<1>, kBufs<1>)
                    : dq(block_dq_simt<2>, kBufs<2>);
  if (s != GATTN_OK) return s;
  return g.D <= 32   ? dkv(block_dkv_simt<0>, kBufs<0>)
         : g.D <= 64 ? dkv(block_dkv_simt<1>, kBufs<1>)
                     : dkv(block_dkv_simt<2>, kBufs<2>);
}

}  // namespace gattn
