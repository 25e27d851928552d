// cache_rows.cu -- rows into the quantised cache, rows back, and block sums of
// what it holds.
//
// Write and read: a lane owns eight elements (one 32-bit word of levels with 4
// bits, two with 8), D / 8 lanes a row, so a warp's load covers whole rows and
// its store whole rows of levels.  A warp stays with one key head and takes
// neighbouring tokens, which lie side by side in the cache.  Everything is read
// and written once: the bound is HBM, next to it the issue slots (about 13
// instructions an element where HBM leaves 14).
//
// Sums: levels are whole numbers, and a step is an 8-bit whole number times a
// power of two, so the sum over a block is one over whole numbers as long as the
// steps and least values of its rows lie within 2^23 of each other: exact in
// 64-bit integers, with one multiply-add an element and no fp64 until the end
// (the GPU adds two fp64 numbers a clock and SM).  Blocks beyond that range are
// summed in fp64, row by row.
#include "cache.cuh"

namespace gattn {

namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <class T>
struct Row8;  // eight elements of a lane
template <>
struct Row8<float> {
  uint4 a, b;
  __device__ void load(const float* x) {
    a = reinterpret_cast<const uint4*>(x)[0];
    b = reinterpret_cast<const uint4*>(x)[1];
  }
  __device__ void get(float* f) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ static void store(float* x, const float* f) {
    reinterpret_cast<float4*>(x)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(x)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Row8<__nv_bfloat16> {
  uint4 a;
  __device__ void load(const __nv_bfloat16* x) { a = *reinterpret_cast<const uint4*>(x); }
  __device__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* x, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(x) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int BITS>
struct Levels;  // of eight elements
template <>
struct Levels<4> {
  using W = uint32_t;
};
template <>
struct Levels<8> {
  using W = uint2;
};

// A row's (m, s) as a pair of bf16, and the levels of the lane's eight elements.
// LPR lanes share the row.
template <int BITS, int LPR>
__device__ __forceinline__ uint32_t quantise(const float* f, typename Levels<BITS>::W* out) {
  constexpr float L = BITS == 4 ? 15.f : 255.f;
  float lo = min_nan(min_nan(min_nan(f[0], f[1]), min_nan(f[2], f[3])),
                     min_nan(min_nan(f[4], f[5]), min_nan(f[6], f[7])));
  float hi = max_nan(max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3])),
                     max_nan(max_nan(f[4], f[5]), max_nan(f[6], f[7])));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  // m: bf16 towards -inf, not below the least finite one
  uint32_t mb = __float_as_uint(lo);
  mb = (int32_t(mb) < 0 ? mb + 0xffffu : mb) & 0xffff0000u;
  if (mb == 0xff800000u) mb = 0xff7f0000u;
  float m = __uint_as_float(mb);
  // s: bf16 towards +inf
  const float st = __fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * m), L / 2);
  uint32_t sb = (__float_as_uint(st) + 0xffffu) & 0xffff0000u;
  if (sb < 0x00800000u) sb = 0;  // below 2^-126
  const float s = __uint_as_float(sb);
  const float inv = sb ? __frcp_rn(s) : 0.f;
  const float c = __fmul_rn(-m, inv);
  // rounding to a whole number: the low bits of t + 1.5 2^23
  constexpr uint32_t kMagic = 0x4b400000u;
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    u[i] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmaf_rn(f[i], inv, c), 0.f), L), 12582912.f));
  uint32_t w0 = 0, w1 = 0;
  if (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w0 += (u[i] - kMagic) << (4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w0 += (u[i] - kMagic) << (8 * i);
      w1 += (u[4 + i] - kMagic) << (8 * i);
    }
  }
  uint32_t par = (mb >> 16) | sb;
  if (!(fabsf(lo) < __int_as_float(0x7f800000) && fabsf(hi) < __int_as_float(0x7f800000))) {
    par = 0x7fc07fc0u;  // a non-finite element: the row is NaN
    w0 = w1 = 0;
  }
  if constexpr (BITS == 4) *out = w0;
  else *out = make_uint2(w0, w1);
  return par;
}

// UN passes of 32 / LPR tokens each for one key head.
template <class T, int BITS, int LPR, int UN>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(const CacheParams p,
                                                                  const T* __restrict__ K,
                                                                  const T* __restrict__ V) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  using W = typename Levels<BITS>::W;
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int64_t w = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int kh = int(w % g.Hkv);
  const int64_t t0 = w / g.Hkv * (RPW * UN);
  if (t0 >= g.Nq) return;
  Row8<T> rk[UN], rv[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int64_t t = min(t0 + u * RPW + sub, int64_t(g.Nq) - 1);
    rk[u].load(K + t * p.ks + kh * D + j * 8);
    rv[u].load(V + t * p.vs + kh * D + j * 8);
  }
  int from = 0;
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int64_t t = t0 + u * RPW + sub;
    int64_t dst = -1;
    if (t < g.Nq) {
      const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, int(t), from);
      if (x.s >= 0) {
        from = x.s;
        const Span sp = span_k(g, x.s);
        const int64_t pos = int64_t(x.i) + sp.len - x.n;
        if (pos >= 0) dst = sp.beg + pos;
      }
    }
    float f[8];
    W wk, wv;
    rk[u].get(f);
    const uint32_t pk = quantise<BITS, LPR>(f, &wk);
    rv[u].get(f);
    const uint32_t pv = quantise<BITS, LPR>(f, &wv);
    if (dst >= 0) {
      const int64_t r = int64_t(kh) * g.Nk + dst;
      reinterpret_cast<W*>(p.k)[r * LPR + j] = wk;
      reinterpret_cast<W*>(p.v)[r * LPR + j] = wv;
      if (j == 0) p.par[r] = make_uint2(pk, pv);
    }
  }
}

// Eight values of a lane
template <int BITS>
__device__ __forceinline__ void values(typename Levels<BITS>::W w, uint32_t par, float* f) {
  const float m = __uint_as_float(par << 16), s = __uint_as_float(par & 0xffff0000u);
  if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a whole number in the low bits of 2^23 + n
      const float n = __uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.f;
      f[i] = __fmaf_rn(s, n, m);
    }
  } else {
    const uint32_t x[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = __uint_as_float(((x[i / 4] >> (8 * (i % 4))) & 255u) | 0x4b000000u) -
                      8388608.f;
      f[i] = __fmaf_rn(s, n, m);
    }
  }
}

template <class T, int BITS, int LPR, int UN>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const CacheParams p,
                                                                 const int32_t* __restrict__ since,
                                                                 T* __restrict__ K,
                                                                 T* __restrict__ V) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  using W = typename Levels<BITS>::W;
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int64_t w = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int kh = int(w % g.Hkv);
  const int64_t t0 = w / g.Hkv * (RPW * UN);
  if (t0 >= g.Nq) return;
  int64_t r[UN];
  int from = 0;
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int64_t t = t0 + u * RPW + sub;
    r[u] = -1;
    if (t < g.Nq) {
      const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, int(t), from);
      if (x.s >= 0) {
        from = x.s;
        const Span sp = span_k(g, x.s);
        const int64_t pos = (since ? int64_t(since[x.s]) : int64_t(sp.len) - x.n) + x.i;
        if (pos >= 0 && pos < sp.len) r[u] = int64_t(kh) * g.Nk + sp.beg + pos;
      }
    }
  }
  W wk[UN], wv[UN];
  uint2 par[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (r[u] >= 0) {
      if (K) wk[u] = reinterpret_cast<const W*>(p.k)[r[u] * LPR + j];
      if (V) wv[u] = reinterpret_cast<const W*>(p.v)[r[u] * LPR + j];
      par[u] = p.par[r[u]];
    }
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (r[u] >= 0) {
      const int64_t o = ((t0 + u * RPW + sub) * g.Hkv + kh) * D + j * 8;
      float f[8];
      if (K) {
        values<BITS>(wk[u], par[u].x, f);
        Row8<T>::store(K + o, f);
      }
      if (V) {
        values<BITS>(wv[u], par[u].y, f);
        Row8<T>::store(V + o, f);
      }
    }
}

// --------------------------------------------------------------------------
// sums
// --------------------------------------------------------------------------
// The whole number v times 2^e in fp64 (|v| < 2^53, v 2^e normal or 0), by integer instructions: the
// conversion instruction runs at the fp64 rate.
__device__ __forceinline__ double scaled(int64_t v, int e) {
  if (v == 0) return 0.0;
  const uint64_t a = v < 0 ? uint64_t(-v) : uint64_t(v);
  const int z = __clzll(a);
  const uint64_t mant = (a << z) >> 11;  // 53 bits, the first set
  const uint64_t bits = (mant & 0xfffffffffffffull) | (uint64_t(1023 + 63 - z + e) << 52) |
                        (v < 0 ? 0x8000000000000000ull : 0);
  return __longlong_as_double(int64_t(bits));
}

// One warp sums one block of one key head: D / 8 lanes a row, 32 / (D / 8)
// rows side by side, their sums joined by shuffles.
template <int BITS, int LPR>
__global__ void __launch_bounds__(kRowThreads) cache_sums_kernel(
    const CacheParams p, const int32_t* __restrict__ since, double* __restrict__ sums, int zs) {
  constexpr int RPW = 32 / LPR, D = LPR * 8, MAXR = kBlkTile / 32;
  using W = typename Levels<BITS>::W;
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int64_t wid = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int kh = int(wid % g.Hkv);
  const int64_t item = wid / g.Hkv;
  int s, b, step = 1, last;
  if (since) {  // warps zs apart share a sequence's blocks from there on
    if (item >= int64_t(g.S) * zs) return;
    s = int(item / zs);
    b = max(since[s], 0) / g.block + int(item % zs);
    step = zs;
    last = (span_k(g, s).len + g.block - 1) / g.block - 1;
  } else {
    if (item >= g.B) return;
    s = piece_seq(g.seq_k, g.S, g.block, int(item));
    b = last = int(item) - piece_base(g.seq_k, s, g.block);
  }
  const Span sp = span_k(g, s);
  const int base = piece_base(g.seq_k, s, g.block);
  for (; b <= last; b += step) {
    const int piece = base + b;
    if (piece < 0 || piece >= g.B) break;
    const int64_t pos = int64_t(b) * g.block;
    const int n = pos >= 0 && pos < sp.len ? int(min(int64_t(g.block), sp.len - pos)) : 0;
    const int64_t r0 = int64_t(kh) * g.Nk + sp.beg + (n ? pos : 0);
    const W* lev = reinterpret_cast<const W*>(p.k) + r0 * LPR + j;
    // exponents of what is not zero: the sums are whole multiples of the least
    uint32_t par[MAXR];
    int emin = 255, emax = 0;
#pragma unroll
    for (int i = 0; i < MAXR; ++i) {
      par[i] = lane + 32 * i < n ? p.par[r0 + lane + 32 * i].x : 0u;
      const int em = (par[i] >> 7) & 255, es = (par[i] >> 23) & 255;
      // a least value below 2^-126 counts as one of that exponent
      if (par[i] & 0x7fffu) emin = min(emin, max(em, 1));
      if (es) emin = min(emin, es);
      emax = max(emax, max(em, es));
    }
    emin = __reduce_min_sync(0xffffffffu, emin);
    emax = __reduce_max_sync(0xffffffffu, emax);
    double* out = sums + (int64_t(piece) * g.Hkv + kh) * D + j * 8;
    if (emax - emin <= 23 && emax < 255) {
      int64_t base_sum = 0;
      uint32_t wt[MAXR];
#pragma unroll
      for (int i = 0; i < MAXR; ++i) {
        const int em = (par[i] >> 7) & 255, es = (par[i] >> 23) & 255;
        const int64_t mm = int64_t((par[i] & 127u) | (em ? 128u : 0u)) << (par[i] & 0x7fffu ? max(em, 1) - emin : 0);
        base_sum += par[i] & 0x8000u ? -mm : mm;
        wt[i] = es ? (((par[i] >> 16) & 127u) | 128u) << (es - emin) : 0u;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) base_sum += __shfl_xor_sync(0xffffffffu, base_sum, o);
      uint64_t a[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = 0;
#pragma unroll
      for (int i = 0; i < MAXR; ++i)
        if (32 * i < n) {
#pragma unroll
          for (int c = 0; c < LPR; c += 4) {  // four rows on their way at a time
            W w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int t = 32 * i + (c + q) * RPW + sub;
              if (t < n) w[q] = lev[int64_t(t) * LPR];
              else w[q] = W{};
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t x = __shfl_sync(0xffffffffu, wt[i], (c + q) * RPW + sub);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                uint32_t u;
                if constexpr (BITS == 4) u = (w[q] >> (4 * k)) & 15u;
                else u = ((k < 4 ? w[q].x : w[q].y) >> (8 * (k % 4))) & 255u;
                a[k] += uint64_t(x) * u;
              }
            }
          }
        }
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] += __shfl_xor_sync(0xffffffffu, a[k], o);
      if (sub == 0) {
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          reinterpret_cast<double2*>(out)[k / 2] =
              make_double2(scaled(int64_t(a[k]) + base_sum, emin - 134),
                           scaled(int64_t(a[k + 1]) + base_sum, emin - 134));
      }
    } else if (sub == 0) {
      double a[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = 0.0;
      for (int t = 0; t < n; ++t) {
        const uint32_t q = p.par[r0 + t].x;
        const double m = __uint_as_float(q << 16), st = __uint_as_float(q & 0xffff0000u);
        const W w = lev[int64_t(t) * LPR];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t u;
          if constexpr (BITS == 4) u = (w >> (4 * k)) & 15u;
          else u = ((k < 4 ? w.x : w.y) >> (8 * (k % 4))) & 255u;
          a[k] += m + st * u;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) out[k] = a[k];
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

template <class T, int BITS, int LPR>
void write_rows(const CacheParams& p, const void* K, const void* V, cudaStream_t st) {
  constexpr int RPW = 32 / LPR, UN = 4;
  const T *k = static_cast<const T*>(K), *v = static_cast<const T*>(V);
  // few rows: a warp for each RPW of them
  const bool few = int64_t(p.g.Nq) * p.g.Hkv < int64_t(sm_count()) * 64 * RPW;
  const int64_t tok = few ? RPW : RPW * UN;
  const int64_t warps = (p.g.Nq + tok - 1) / tok * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  if (few) cache_write_kernel<T, BITS, LPR, 1><<<grid, kRowThreads, 0, st>>>(p, k, v);
  else cache_write_kernel<T, BITS, LPR, UN><<<grid, kRowThreads, 0, st>>>(p, k, v);
}

template <class T, int BITS, int LPR>
void read_rows(const CacheParams& p, const int32_t* since, void* K, void* V, cudaStream_t st) {
  constexpr int RPW = 32 / LPR, UN = 4;
  const bool few = int64_t(p.g.Nq) * p.g.Hkv < int64_t(sm_count()) * 64 * RPW;
  const int64_t tok = few ? RPW : RPW * UN;
  const int64_t warps = (p.g.Nq + tok - 1) / tok * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
  if (few) cache_read_kernel<T, BITS, LPR, 1><<<grid, kRowThreads, 0, st>>>(p, since, k, v);
  else cache_read_kernel<T, BITS, LPR, UN><<<grid, kRowThreads, 0, st>>>(p, since, k, v);
}

// f(type, bits, lanes per row)
template <class F>
void by_layout(const CacheParams& p, F f) {
  const auto lanes = [&](auto bits) {
    if (p.g.D == 32) f(bits, std::integral_constant<int, 4>{});
    else if (p.g.D == 64) f(bits, std::integral_constant<int, 8>{});
    else f(bits, std::integral_constant<int, 16>{});
  };
  if (p.bits == 4) lanes(std::integral_constant<int, 4>{});
  else lanes(std::integral_constant<int, 8>{});
}

}  // namespace

gattn_status launch_cache_write(const CacheParams& p, gattn_dtype dt, const void* K, const void* V,
                                cudaStream_t st) {
  by_layout(p, [&](auto bits, auto lpr) {
    if (dt == GATTN_F32) write_rows<float, bits(), lpr()>(p, K, V, st);
    else write_rows<__nv_bfloat16, bits(), lpr()>(p, K, V, st);
  });
  return launched("gattn_cache_write");
}

gattn_status launch_cache_read(const CacheParams& p, gattn_dtype dt, const int32_t* since, void* K,
                               void* V, cudaStream_t st) {
  by_layout(p, [&](auto bits, auto lpr) {
    if (dt == GATTN_F32) read_rows<float, bits(), lpr()>(p, since, K, V, st);
    else read_rows<__nv_bfloat16, bits(), lpr()>(p, since, K, V, st);
  });
  return launched("gattn_cache_read");
}

gattn_status launch_cache_sums(const CacheParams& p, const int32_t* since, double* sums,
                               cudaStream_t st) {
  // since: as many warps to a sequence as blocks of it would fill the GPU, since a call may renew
  // one block of each or all of one
  int zs = 1;
  while (since && zs < 64 && int64_t(zs) * p.g.S * p.g.Hkv < int64_t(sm_count()) * 32 &&
         int64_t(zs) * p.g.block < p.g.Nk)
    zs *= 2;
  const int64_t warps = (since ? int64_t(p.g.S) * zs : int64_t(p.g.B)) * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  by_layout(p, [&](auto bits, auto lpr) {
    cache_sums_kernel<bits(), lpr()><<<grid, kRowThreads, 0, st>>>(p, since, sums, zs);
  });
  return launched("gattn_cache_sums");
}

}  // namespace gattn
