// block_simt.cu -- block attention on the CUDA cores, for fp32 tensors (the
// tensor cores' kinds keep fewer than 24 bits of a product's operands).
//
// 64 x 64 score tiles in fp32: 256 threads hold 4 x 4 scores each, operands
// are staged in shared memory as fp32, and a thread's 4 rows of the output
// (or gradient) stay in registers.  Bound by the FMA units: a step of 64
// rows by 64 keys is 2 (forward), 3 (dQ) or 4 (dK, dV) products of
// 64 x 64 x D.
//
// With the unit's block list ascending, the keys a row may see are the first
// columns of its steps, so the mask of a row is one number (list_keys).
#include <algorithm>

#include "attn_launch.cuh"
#include "block.cuh"

namespace gattn {

namespace {

constexpr int kR = 64;     // rows of a tile
constexpr int kC = 64;     // keys of a step
constexpr int kThr = 256;
constexpr int kPS = kC + 4;  // row stride of the score tile

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

struct FwdP {
  BlockGeom g;
  const void *Q, *K, *V;
  const int32_t* idx;
  void* out;
  float* lse;
};

// element offset of the (row, head) pair r of a unit, -1 past its rows
__device__ __forceinline__ int64_t q_off(const BlockGeom& g, const Unit& u, int kh, int r) {
  const int t = r / g.G;
  if (t >= u.n) return -1;
  return (int64_t(u.row + t) * g.H + kh * g.G + (r - t * g.G)) * g.D;
}

// 64 rows of D elements to shared memory (row stride D + 4); off(r) < 0: zeros
template <class T, class F>
__device__ __forceinline__ void stage(float* dst, const T* src, int D, F off) {
  const int ld = D + 4;
  for (int i = threadIdx.x; i < kR * D; i += kThr) {
    const int r = i / D, d = i - r * D;
    const int64_t o = off(r);
    dst[r * ld + d] = o >= 0 ? to_f(src[o + d]) : 0.f;
  }
}

// s[i][j] = a[4 ty + i] . b[tx + 16 j]
__device__ __forceinline__ void dots(const float* a, const float* b, int D, float s[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ld = D + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
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

// o[i][*] += sum_k w(4 ty + i, k) b[k][cols of this thread], cols 4 tx + 64 q.
// TR: w is stored [k][row].  GUARD: a zero weight takes nothing from its row
// of b, which may hold non-finite values that the row must not see.
template <int DQ, bool TR, bool GUARD>
__device__ __forceinline__ void weighted(const float* w, const float* b, int D, float o[4][DQ][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ld = D + 4;
  for (int k = 0; k < kC; ++k) {
    float x[4];
    if (TR) {
      const float4 v = *reinterpret_cast<const float4*>(w + k * kPS + ty * 4);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[(ty * 4 + i) * kPS + k];
    }
#pragma unroll
    for (int q = 0; q < DQ; ++q) {
      const int c = tx * 4 + 64 * q;
      if (c < D) {
        const float4 v = *reinterpret_cast<const float4*>(b + k * ld + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (GUARD && x[i] == 0.f) continue;
          o[i][q][0] = fmaf(x[i], v.x, o[i][q][0]);
          o[i][q][1] = fmaf(x[i], v.y, o[i][q][1]);
          o[i][q][2] = fmaf(x[i], v.z, o[i][q][2]);
          o[i][q][3] = fmaf(x[i], v.w, o[i][q][3]);
        }
      }
    }
  }
}

template <class T, int DQ>
__device__ __forceinline__ void put4(T* p, const float* v, float mul) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = from_f<T>(v[e] * mul);
}

// key row (element offset of K, V) of column c of the step that starts at
// list key k0, -1 past the list
__device__ __forceinline__ int64_t k_off(const BlockGeom& g, const int* ids, int total, int k0,
                                         int c, int kbeg, int kh) {
  const int k = k0 + c;
  if (k >= total) return -1;
  return (int64_t(kbeg + ids[k / g.block] * g.block + k % g.block) * g.Hkv + kh) * g.D;
}

template <class T, int DQ>
__global__ void __launch_bounds__(kThr) block_fwd_simt(const FwdP p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int ids[kBlkMaxTopk];
  __shared__ int n_ids;
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4, kh = blockIdx.y, u = blockIdx.x, r0 = blockIdx.z * kR;
  float *sQ = sm, *sK = sQ + kR * ld, *sV = sK + kC * ld, *sP = sV + kC * ld;
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
  const T* K = static_cast<const T*>(p.K);
  const T* V = static_cast<const T*>(p.V);
  stage(sQ, static_cast<const T*>(p.Q), D, [&](int r) { return q_off(g, un, kh, r0 + r); });
  float m[4], l[4], o[4][DQ][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = neg_inf();
    l[i] = 0.f;
#pragma unroll
    for (int q = 0; q < DQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][q][e] = 0.f;
  }
  for (int k0 = 0; k0 < total; k0 += kC) {
    __syncthreads();
    auto off = [&](int c) { return k_off(g, ids, total, k0, c, ks.beg, kh); };
    stage(sK, K, D, off);
    stage(sV, V, D, off);
    __syncthreads();
    float s[4][4];
    dots(sQ, sK, D, s);
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
      for (int q = 0; q < DQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][q][e] *= corr;
    }
    __syncwarp();  // a row's weights come from the half-warp that uses them
    if (k0 + kC > lim0) weighted<DQ, false, true>(sP, sV, D, o);
    else weighted<DQ, false, false>(sP, sV, D, o);
  }
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = q_off(g, un, kh, r0 + ty * 4 + i);
    if (at < 0) continue;
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    if (tx == 0) p.lse[at / D] = l[i] != 0.f ? (m[i] + lg2(l[i])) * kLn2 : neg_inf();
#pragma unroll
    for (int q = 0; q < DQ; ++q) {
      const int c = tx * 4 + 64 * q;
      if (c < D) put4<T, DQ>(out + at + c, o[i][q], inv);
    }
  }
}

// dQ of 64 (row, head) pairs of a unit
template <class T, int DQ>
__global__ void __launch_bounds__(kThr) block_dq_simt(const BlockBwdParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int ids[kBlkMaxTopk];
  __shared__ int n_ids;
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4, kh = blockIdx.y, u = blockIdx.x, r0 = blockIdx.z * kR;
  float *sQ = sm, *sO = sQ + kR * ld, *sK = sO + kR * ld, *sV = sK + kC * ld, *sP = sV + kC * ld;
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
  float L[4], Dl[4], o[4][DQ][4];
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
    for (int q = 0; q < DQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][q][e] = 0.f;
  }
  const auto qo = [&](int r) { return q_off(g, un, kh, r0 + r); };
  stage(sQ, static_cast<const T*>(p.Q), D, qo);
  stage(sO, static_cast<const T*>(p.dO), D, qo);
  for (int k0 = 0; k0 < total; k0 += kC) {
    __syncthreads();
    auto off = [&](int c) { return k_off(g, ids, total, k0, c, ks.beg, kh); };
    stage(sK, static_cast<const T*>(p.K), D, off);
    stage(sV, static_cast<const T*>(p.V), D, off);
    __syncthreads();
    float s[4][4], dp[4][4];
    dots(sQ, sK, D, s);
    dots(sO, sV, D, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = k0 + tx + 16 * j < lim[i];
        const float w = in ? ex2(fmaf(s[i][j], g.qmul, -L[i])) * (dp[i][j] - Dl[i]) : 0.f;
        sP[(ty * 4 + i) * kPS + tx + 16 * j] = w;
      }
    __syncwarp();
    weighted<DQ, false, false>(sP, sK, D, o);
  }
  T* dQ = static_cast<T*>(p.dQ);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = q_off(g, un, kh, r0 + ty * 4 + i);
    if (at < 0) continue;
#pragma unroll
    for (int q = 0; q < DQ; ++q) {
      const int c = tx * 4 + 64 * q;
      if (c < D) put4<T, DQ>(dQ + at + c, o[i][q], g.scale);
    }
  }
}

// dK, dV of one half (64 keys) of a work item's key tile
template <class T, int DQ>
__global__ void __launch_bounds__(kThr) block_dkv_simt(const BlockBwdParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int list[1024];
  __shared__ uint8_t mask[1024];
  __shared__ int n_list, n_all;
  const BlockGeom& g = p.g;
  const int D = g.D, ld = D + 4;
  float *sK = sm, *sV = sK + kC * ld, *sQ = sV + kC * ld, *sO = sQ + kR * ld, *sP = sO + kR * ld;
  float* sS = sP + kR * kPS;
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
    stage(sK, static_cast<const T*>(p.K), D, ko);
    stage(sV, static_cast<const T*>(p.V), D, ko);
    float gk[4][DQ][4], gv[4][DQ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < DQ; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) gk[i][x][e] = gv[i][x][e] = 0.f;
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
      for (int e = 0; e < nl; ++e) {
        const int u = list[e];
        const uint32_t mk = mask[e];
        const int64_t uo = int64_t(u - ub) * g.qb;
        if (uo < 0 || uo >= qs.len) continue;  // only where offsets lie about the tables
        Unit un;
        un.s = s;
        un.row = qs.beg + int(uo);
        un.n = min(g.qb, qs.len - int(uo));
        un.pos = int(uo) + ks.len - qs.len;
        for (int r0 = 0; r0 < un.n * g.G; r0 += kR) {
          __syncthreads();
          const auto qo = [&](int r) { return q_off(g, un, kh, r0 + r); };
          stage(sQ, static_cast<const T*>(p.Q), D, qo);
          stage(sO, static_cast<const T*>(p.dO), D, qo);
          __syncthreads();
          float sc[4][4], dp[4][4];
          dots(sQ, sK, D, sc);
          dots(sO, sV, D, dp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + ty * 4 + i, t = r / g.G;
            const int64_t at = q_off(g, un, kh, r);
            const float2 stat = at >= 0 ? p.stat[at / D] : make_float2(0.f, 0.f);
            const int end = at < 0 ? 0 : g.causal ? min(un.pos + t + 1, ks.len) : ks.len;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = tx + 16 * j, pos = pos0 + c;
              const bool in = pos < end && ((mk >> ((half * kC + c) / g.block)) & 1u);
              const float w = in ? ex2(fmaf(sc[i][j], g.qmul, -stat.x)) : 0.f;
              sP[(ty * 4 + i) * kPS + c] = w;
              sS[(ty * 4 + i) * kPS + c] = in ? w * (dp[i][j] - stat.y) : 0.f;
            }
          }
          __syncthreads();
          weighted<DQ, true, false>(sP, sO, D, gv);
          weighted<DQ, true, false>(sS, sQ, D, gk);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = ty * 4 + i;
      const int64_t at = ko(c);
      if (at < 0) continue;
#pragma unroll
      for (int x = 0; x < DQ; ++x) {
        const int d = tx * 4 + 64 * x;
        if (d >= D) continue;
        if (q.w < 0) {
          put4<T, DQ>(static_cast<T*>(p.dK) + at + d, gk[i][x], g.scale);
          put4<T, DQ>(static_cast<T*>(p.dV) + at + d, gv[i][x], 1.f);
        } else {
          float* o = p.part + (int64_t(q.w) * 2 * kBlkTile + half * kC + c) * D + d;
          *reinterpret_cast<float4*>(o) =
              make_float4(gk[i][x][0], gk[i][x][1], gk[i][x][2], gk[i][x][3]);
          *reinterpret_cast<float4*>(o + int64_t(kBlkTile) * D) =
              make_float4(gv[i][x][0], gv[i][x][1], gv[i][x][2], gv[i][x][3]);
        }
      }
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

template <class T>
gattn_status fwd(const FwdP& p, dim3 grid, cudaStream_t st) {
  const int fl = 3 * kR * (p.g.D + 4) + kR * kPS;
  return p.g.D > 64 ? go(block_fwd_simt<T, 2>, grid, fl, p, st, "gattn_block_fwd")
                    : go(block_fwd_simt<T, 1>, grid, fl, p, st, "gattn_block_fwd");
}

template <class T>
gattn_status bwd(const BlockBwdParams& p, dim3 grid, cudaStream_t st) {
  const int fl = 4 * kR * (p.g.D + 4) + kR * kPS, fk = fl + kR * kPS;
  const dim3 gk(unsigned(std::min<int64_t>(2 * p.max_items, int64_t(sm_count()) * 2)));
  gattn_status s = GATTN_OK;
  if (p.g.U > 0)
    s = p.g.D > 64 ? go(block_dq_simt<T, 2>, grid, fl, p, st, "gattn_block_bwd (dQ)")
                   : go(block_dq_simt<T, 1>, grid, fl, p, st, "gattn_block_bwd (dQ)");
  if (s != GATTN_OK) return s;
  return p.g.D > 64 ? go(block_dkv_simt<T, 2>, gk, fk, p, st, "gattn_block_bwd (dK, dV)")
                    : go(block_dkv_simt<T, 1>, gk, fk, p, st, "gattn_block_bwd (dK, dV)");
}

dim3 row_grid(const BlockGeom& g) {
  return dim3(unsigned(g.U), unsigned(g.Hkv), unsigned((g.qb * g.G + kR - 1) / kR));
}

}  // namespace

gattn_status launch_block_fwd_simt(const BlockGeom& g, gattn_dtype dt, const void* Q,
                                   const void* K, const void* V, const int32_t* idx, void* out,
                                   float* lse, cudaStream_t st) {
  const FwdP p{g, Q, K, V, idx, out, lse};
  return dt == GATTN_F32 ? fwd<float>(p, row_grid(g), st) : fwd<__nv_bfloat16>(p, row_grid(g), st);
}

gattn_status launch_block_bwd_simt(const BlockBwdParams& p, gattn_dtype dt, cudaStream_t st) {
  return dt == GATTN_F32 ? bwd<float>(p, row_grid(p.g), st)
                         : bwd<__nv_bfloat16>(p, row_grid(p.g), st);
}

}  // namespace gattn
