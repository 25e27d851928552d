// cache_rows.cu -- rows into the quantised cache, rows back, and block sums of
// what it holds.
//
// Write and read: a lane owns eight elements (one 32-bit word of levels with 4
// bits, two with 8), D / 8 lanes a row, so a warp's load covers whole rows and
// its store whole rows of levels.  A warp stays with one key head and takes
// neighbouring tokens, which lie side by side in the cache.  Everything is read
// and written once: the bound is HBM, next to it the issue slots.  What is
// formed once a row (bounds, step, place in the cache) is formed by one lane: the
// lanes of a row hold eight rows (K and V of four tokens) and reduce them so that each
// lane ends with rows of its own.
//
// Sums: sum (m + s u) over a block is sum m plus sum s u, and the second is a
// product of levels with a vector: tensor cores, as in the attention (levels are
// fp16 whole numbers as they lie).  Steps have 8 bits and levels 4 or 8, so the
// fp32 sums of 64 rows are exact as long as the steps' exponents are within 6 (2 with 8
// bits) of each other, of 128 within one less: the eight columns of a product take a class
// of exponents each.  Blocks beyond all classes are summed in fp64, row by row.
//
// Measured: 32,768 rows of 8 heads of 128 in bf16 written in 31 us (170 MB, 5.5 TB/s) and read back in 27
// (6.3 TB/s), issue slots 70% busy in both; 31,700 rows read in 25.6; 65,544 rows of 8 heads of 64
// summed in 9.2 us (2.7 TB/s), where 600 instructions to a block of 64 rows are the bound.
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
  float f[8];
  // wide: rows start on 32-byte borders, one instruction
  __device__ void load(const float* x, bool wide) {
    if (wide) {
      asm volatile("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                   : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]),
                     "=f"(f[6]), "=f"(f[7])
                   : "l"(x));
    } else {
      const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
  }
  __device__ void get(float* to) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) to[i] = f[i];
  }
  __device__ static void store(float* x, const float* f, bool wide) {
    if (wide) {
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(x), "f"(f[0]),
                   "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                   : "memory");
    } else {
      reinterpret_cast<float4*>(x)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(x)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
};
template <>
struct Row8<__nv_bfloat16> {
  uint4 a;
  __device__ void load(const __nv_bfloat16* x, bool) { a = *reinterpret_cast<const uint4*>(x); }
  __device__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* x, const float* f, bool) {
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

// least element and minus the greatest, NaN if there is one
template <class T>
struct Bounds;
template <>
struct Bounds<float> {
  float lo, nhi;
  __device__ static Bounds of(const Row8<float>& r) {
    float f[8];
    r.get(f);
    return {min_nan(min_nan(min_nan(f[0], f[1]), min_nan(f[2], f[3])),
                    min_nan(min_nan(f[4], f[5]), min_nan(f[6], f[7]))),
            -max_nan(max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3])),
                     max_nan(max_nan(f[4], f[5]), max_nan(f[6], f[7])))};
  }
  __device__ Bounds from(int o) const {
    return {__shfl_xor_sync(0xffffffffu, lo, o), __shfl_xor_sync(0xffffffffu, nhi, o)};
  }
  __device__ void join(Bounds x) {
    lo = min_nan(lo, x.lo);
    nhi = min_nan(nhi, x.nhi);
  }
  __device__ float least() const { return lo; }
  __device__ float greatest() const { return -nhi; }
};
template <>
struct Bounds<__nv_bfloat16> {
  uint32_t z;  // both as bf16
  __device__ static uint32_t least2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static uint32_t greatest2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static Bounds of(const Row8<__nv_bfloat16>& r) {
    const uint32_t lo = least2(least2(r.a.x, r.a.y), least2(r.a.z, r.a.w));
    const uint32_t hi = greatest2(greatest2(r.a.x, r.a.y), greatest2(r.a.z, r.a.w)) ^ 0x80008000u;
    return {least2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632))};
  }
  __device__ Bounds from(int o) const { return {__shfl_xor_sync(0xffffffffu, z, o)}; }
  __device__ void join(Bounds x) { z = least2(z, x.z); }
  __device__ float least() const { return __uint_as_float(z << 16); }
  __device__ float greatest() const { return -__uint_as_float(z & 0xffff0000u); }
};

// (m, s) of a row as a pair of bf16, and the factors of its levels
struct Steps {
  uint32_t par;
  float inv, c;
  bool clamp;  // levels may leave [0, L], or the row is not finite
};
template <int BITS>
__device__ __forceinline__ Steps steps(float lo, float hi) {
  constexpr float L = BITS == 4 ? 15.f : 255.f;
  // m: bf16 towards -inf, not below the least finite one
  uint32_t mb = __float_as_uint(lo);
  mb = (int32_t(mb) < 0 ? mb + 0xffffu : mb) & 0xffff0000u;
  const bool lowest = mb == 0xff800000u;  // elements may be less than m then
  if (lowest) mb = 0xff7f0000u;
  const float m = __uint_as_float(mb);
  // s: bf16 towards +inf
  const float st = __fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * m), L / 2);
  uint32_t sb = (__float_as_uint(st) + 0xffffu) & 0xffff0000u;
  if (sb < 0x00800000u) sb = 0;  // below 2^-126
  Steps r;
  r.inv = sb ? __frcp_rn(__uint_as_float(sb)) : 0.f;
  r.c = __fmul_rn(-m, r.inv);
  r.par = (mb >> 16) | sb;
  // c is rounded to 2^-24 of its size: below 2^21 that is less than a quarter of a level
  r.clamp = lowest || !(fabsf(r.c) < 2097152.f);
  if (!(fabsf(lo) < __int_as_float(0x7f800000) && fabsf(hi) < __int_as_float(0x7f800000))) {
    r.par = 0x7fc07fc0u;  // a non-finite element: the row is NaN, its levels 0
    r.inv = r.c = 0.f;
    r.clamp = true;
  }
  return r;
}

template <int BITS, bool CLAMP>
__device__ __forceinline__ typename Levels<BITS>::W levels(const float* f, float inv, float c) {
  constexpr float L = BITS == 4 ? 15.f : 255.f;
  // rounding to a whole number: the low bits of t + 1.5 2^23
  constexpr uint32_t kMagic = 0x4b400000u;
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t = __fmaf_rn(f[i], inv, c);
    if (CLAMP) t = fminf(fmaxf(t, 0.f), L);
    u[i] = __float_as_uint(__fadd_rn(t, 12582912.f)) - kMagic;
  }
  if constexpr (BITS == 4) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w += u[i] << (4 * i);
    return w;
  } else {
    uint32_t w0 = 0, w1 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w0 += u[i] << (8 * i);
      w1 += u[4 + i] << (8 * i);
    }
    return make_uint2(w0, w1);
  }
}

// Tokens t0 + u * (32 / LPR) + (the lane's group), u < UN, for one key head.  Row 2u of a group is
// K of token u, row 2u + 1 V.
template <class T, int BITS, int LPR, int UN>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(const CacheParams p,
                                                                  const T* __restrict__ K,
                                                                  const T* __restrict__ V,
                                                                  bool wide) {
  constexpr int RPW = 32 / LPR, D = LPR * 8, NR = 2 * UN;
  constexpr int OWN = NR > LPR ? NR / LPR : 1;  // rows of a lane in the end
  using W = typename Levels<BITS>::W;
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int64_t w = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int kh = int(w) & (g.Hkv - 1);  // a power of two
  const int64_t t0 = (w >> (31 - __clz(g.Hkv))) * (RPW * UN) + sub;
  if (t0 - sub >= g.Nq) return;
  Row8<T> row[NR];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int64_t t = min(t0 + u * RPW, int64_t(g.Nq) - 1);
    row[2 * u].load(K + t * p.ks + kh * D + j * 8, wide);
    row[2 * u + 1].load(V + t * p.vs + kh * D + j * 8, wide);
  }
  // where the lane's own rows go, while they are on their way
  const int first = j * NR / LPR;
  int dst[OWN];
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    const int64_t t = t0 + (first + o) / 2 * RPW;
    dst[o] = -1;
    if (t < g.Nq) {
      const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, int(t));
      if (x.s >= 0) {
        const Span sp = span_k(g, x.s);
        const int pos = x.i + sp.len - x.n;  // within +-2^31: all three are row counts
        if (pos >= 0) dst[o] = sp.beg + pos;
      }
    }
  }
  Bounds<T> b[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) b[r] = Bounds<T>::of(row[r]);
  int n = NR;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    if (n > 1) {  // keep one half of the rows, give the other
      n /= 2;
      const bool up = j & o;
#pragma unroll
      for (int r = 0; r < NR / 2; ++r)
        if (r < n) {
          Bounds<T> keep = up ? b[r + n] : b[r];
          const Bounds<T> give = up ? b[r] : b[r + n];
          keep.join(give.from(o));
          b[r] = keep;
        }
    } else {
      b[0].join(b[0].from(o));
    }
  }
  Steps st[OWN];
  bool clamp = false;
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    st[o] = steps<BITS>(b[o].least(), b[o].greatest());
    clamp = clamp || st[o].clamp;
    // lanes that share a row write it alike
    if (dst[o] >= 0)
      reinterpret_cast<uint32_t*>(p.par)[(int64_t(kh) * g.Nk + dst[o]) * 2 + ((first + o) & 1)] =
          st[o].par;
  }
  clamp = __any_sync(0xffffffffu, clamp);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int from = r * LPR / NR, o = OWN > 1 ? r % OWN : 0;
    const float inv = __shfl_sync(0xffffffffu, st[o].inv, from, LPR);
    const float c = __shfl_sync(0xffffffffu, st[o].c, from, LPR);
    const int to = __shfl_sync(0xffffffffu, dst[o], from, LPR);
    float f[8];
    row[r].get(f);
    const W lev = clamp ? levels<BITS, true>(f, inv, c) : levels<BITS, false>(f, inv, c);
    if (to >= 0)
      reinterpret_cast<W*>(r & 1 ? p.v : p.k)[(int64_t(kh) * g.Nk + to) * LPR + j] = lev;
  }
}

// Eight values of a lane.  A level, masked in place and put into the low bits of
// 2^23, is a whole number times 16^i (256^i); the factor is taken out of the step.
template <int BITS>
__device__ __forceinline__ void values(typename Levels<BITS>::W w, uint32_t par, float* f) {
  const float m = __uint_as_float(par << 16), s = __uint_as_float(par & 0xffff0000u);
  if constexpr (BITS == 4) {
    const float sc[4] = {s, s * 0x1p-4f, s * 0x1p-8f, s * 0x1p-12f};
    const uint32_t half[2] = {w, w >> 16};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = __uint_as_float((half[i / 4] & (15u << (4 * (i % 4)))) | 0x4b000000u);
      f[i] = __fmaf_rn(sc[i % 4], n - 8388608.f, m);
    }
  } else {
    const uint32_t x[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = __uint_as_float(__byte_perm(x[i / 4], 0x4b000000u, 0x7440 + i % 4));
      f[i] = __fmaf_rn(s, n - 8388608.f, m);
    }
  }
}

template <class T, int BITS, int LPR, int UN>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const CacheParams p,
                                                                 const int32_t* __restrict__ since,
                                                                 T* __restrict__ K,
                                                                 T* __restrict__ V, bool wide) {
  constexpr int RPW = 32 / LPR, D = LPR * 8;
  static_assert(UN <= LPR, "a lane finds one token's row");
  using W = typename Levels<BITS>::W;
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, sub = lane / LPR, j = lane % LPR;
  const int64_t w = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int kh = int(w) & (g.Hkv - 1);  // a power of two
  const int64_t t0 = (w >> (31 - __clz(g.Hkv))) * (RPW * UN) + sub;
  if (t0 - sub >= g.Nq) return;
  int mine = -1;
  {
    const int64_t t = t0 + j % UN * RPW;
    if (t < g.Nq) {
      const SeqRow x = seq_row(g.seq_q, g.S, g.Nq, int(t));
      if (x.s >= 0) {
        const Span sp = span_k(g, x.s);
        const int64_t pos = (since ? int64_t(since[x.s]) : int64_t(sp.len) - x.n) + x.i;
        if (pos >= 0 && pos < sp.len) mine = sp.beg + int(pos);
      }
    }
  }
  W wk[UN], wv[UN];
  uint2 par[UN];
  int r[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    r[u] = __shfl_sync(0xffffffffu, mine, u, LPR);
    if (r[u] >= 0) {
      const int64_t at = int64_t(kh) * g.Nk + r[u];
      if (K) wk[u] = reinterpret_cast<const W*>(p.k)[at * LPR + j];
      if (V) wv[u] = reinterpret_cast<const W*>(p.v)[at * LPR + j];
      par[u] = p.par[at];
    }
  }
  const int64_t out = (t0 * g.Hkv + kh) * D + j * 8, step = int64_t(RPW) * g.Hkv * D;
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (r[u] >= 0) {
      float f[8];
      if (K) {
        values<BITS>(wk[u], par[u].x, f);
        Row8<T>::store(K + out + u * step, f, wide);
      }
      if (V) {
        values<BITS>(wv[u], par[u].y, f);
        Row8<T>::store(V + out + u * step, f, wide);
      }
    }
}

// --------------------------------------------------------------------------
// sums
// --------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// x 2^e in fp64 (x is 0 or normal, the result normal), by integer instructions: the conversion
// instruction runs at the fp64 rate, two a clock and SM
__device__ __forceinline__ double widened(float x, int e) {
  const uint32_t b = __float_as_uint(x);
  if (b == 0) return 0.0;
  return __hiloint2double(int(((b >> 3) & 0x0fffffffu) + (uint32_t(896 + e) << 20)), int(b << 29));
}
// the whole number v (of at most 53 bits) times 2^e, 0 or normal
__device__ __forceinline__ double scaled(int64_t v, int e) {
  const double x = __ll2double_rn(v);
  return v == 0 ? 0.0 : __hiloint2double(__double2hiint(x) + e * 0x100000, __double2loint(x));
}

// One warp sums one block (of at most NR rows) of one key head: 16 rows a product, of which a lane
// holds D / 8 levels of four.
template <int BITS, int D, int NR>
__global__ void __launch_bounds__(kRowThreads, D * BITS > 512 ? 2 : D * BITS > 256 ? 3 : 4) cache_sums_kernel(
    const CacheParams p, const int32_t* __restrict__ since, double* __restrict__ sums, int lz) {
  constexpr int RB = D * BITS / 8, VB = RB / 8, VW = VB < 4 ? 1 : VB / 4, MT = D / 16;
  constexpr int CH = VB == 16 || NR == 32 ? 2 : 4;  // 16-row pieces on their way at a time
  // exponents of a class: with 8 bits of the step, those of a level and of the rows, 24 together
  constexpr int kClass = 16 - BITS - (NR > 64 ? 7 : 6);
  constexpr int kSpread = 8 * kClass < 29 ? 8 * kClass : 29;  // 24 bits and the classes in 53
  __shared__ __align__(16) uint16_t weight[kRowThreads / 32][NR];
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
  // all divisors are powers of two
  const int lb = 31 - __clz(g.block), lh = 31 - __clz(g.Hkv);
  const int64_t wid = int64_t(blockIdx.x) * (kRowThreads / 32) + warp;
  const int kh = int(wid) & (g.Hkv - 1);
  const int64_t item = wid >> lh;
  const auto base_of = [&](int i) { return (max(g.seq_k[i], 0) >> lb) + i; };  // piece_base
  int s, b, step = 1, last;
  if (since) {  // 2^lz warps share a sequence's blocks from there on
    if (item >> lz >= g.S) return;
    s = int(item >> lz);
    b = (max(since[s], 0) >> lb) + (int(item) & ((1 << lz) - 1));
    step = 1 << lz;
    last = ((span_k(g, s).len + g.block - 1) >> lb) - 1;
  } else {
    if (item >= g.B) return;
    int lo = 0;
    for (int n = g.S; n > 1;) {  // piece_seq
      const int st = (n + 31) >> 5, i = lo + lane * st;
      const unsigned m = __ballot_sync(0xffffffffu, i < lo + n && base_of(i) <= int(item));
      const int hi = m ? 31 - __clz(m) : 0;
      n = min(st, n - hi * st);
      lo += hi * st;
    }
    s = lo;
    b = last = int(item) - base_of(s);
  }
  const Span sp = span_k(g, s);
  const int base = base_of(s);
  for (; b <= last; b += step) {
    const int piece = base + b;
    if (piece < 0 || piece >= g.B) break;
    const int64_t pos = int64_t(b) << lb;
    const int n = pos >= 0 && pos < sp.len ? int(min(int64_t(g.block), sp.len - pos)) : 0;
    const int64_t r0 = int64_t(kh) * g.Nk + sp.beg + (n ? pos : 0);
    double* out = sums + (int64_t(piece) * g.Hkv + kh) * D;
    uint32_t par[NR / 32];
#pragma unroll
    for (int i = 0; i < NR / 32; ++i)
      par[i] = lane + 32 * i < n ? p.par[r0 + lane + 32 * i].x : 0u;
    // levels of 16 CH rows are on their way while the exponents are looked at
    const uint8_t* lev = p.k + (r0 + 2 * t) * RB + gq * VB;
    uint32_t v[CH][4][VW];
    const auto fetch = [&](int at) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = at + 16 * c + 8 * (q >> 1) + (q & 1);
          const uint8_t* a = lev + r * RB;
#pragma unroll
          for (int w = 0; w < VW; ++w) v[c][q][w] = 0;
          if (r + 2 * t < n) {
            if constexpr (VB == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(a);
              v[c][q][0] = x.x; v[c][q][1] = x.y; v[c][q][2] = x.z; v[c][q][3] = x.w;
            } else if constexpr (VB == 8) {
              const uint2 x = *reinterpret_cast<const uint2*>(a);
              v[c][q][0] = x.x; v[c][q][1] = x.y;
            } else if constexpr (VB == 4) {
              v[c][q][0] = *reinterpret_cast<const uint32_t*>(a);
            } else {
              v[c][q][0] = *reinterpret_cast<const uint16_t*>(a);
            }
          }
        }
    };
    fetch(0);
    // exponents of the steps and of the least values (one below 2^-126 counts as that)
    int se = 255, sx = 0, me = 255, mx = 0;
#pragma unroll
    for (int i = 0; i < NR / 32; ++i) {
      const int em = (par[i] >> 7) & 255, es = (par[i] >> 23) & 255;
      if (par[i] & 0x7fffu) me = min(me, max(em, 1));
      mx = max(mx, em);
      if (es) se = min(se, es);
      sx = max(sx, es);
    }
    se = __reduce_min_sync(0xffffffffu, se);
    sx = __reduce_max_sync(0xffffffffu, sx);
    me = __reduce_min_sync(0xffffffffu, me);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (sx - se >= kSpread || sx == 255 || mx == 255 || mx - me > 38) {
      for (int d = lane; d < D; d += 32) {
        double a = 0.0;
#pragma unroll 4
        for (int r = 0; r < n; ++r) {
          const uint32_t q = p.par[r0 + r].x;
          const uint32_t w = p.k[(r0 + r) * RB + d * BITS / 8];
          const uint32_t u = BITS == 4 ? (w >> (d % 2 * 4)) & 15u : w;
          a += double(__uint_as_float(q << 16)) + double(__uint_as_float(q & 0xffff0000u)) * u;
        }
        out[d] = a;
      }
      continue;
    }
    // least values: whole multiples of 2^(me - 134)
    int64_t msum = 0;
#pragma unroll
    for (int i = 0; i < NR / 32; ++i) {
      const int em = (par[i] >> 7) & 255;
      const int64_t x = int64_t((par[i] & 127u) | (em ? 128u : 0u))
                        << (par[i] & 0x7fffu ? max(em, 1) - me : 0);
      msum += par[i] & 0x8000u ? -x : x;
    }
    if (mx - me <= 15) {
      msum = __reduce_add_sync(0xffffffffu, int(msum));  // 128 rows of 2^23
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) msum += __shfl_xor_sync(0xffffffffu, msum, o);
    }
    // Steps in fp16, as multiples of 2^(se + class kClass - 127); with several classes, the class in
    // what that leaves free: an exponent below kClass takes three of the five bits.
    const bool one = sx - se < kClass;
#pragma unroll
    for (int i = 0; i < NR / 32; ++i) {
      const uint32_t es = (par[i] >> 23) & 255, mant = (par[i] >> 13) & 0x3f8u;
      const int k = int(es) - se, cls = max(k, 0) / kClass;
      weight[warp][lane + 32 * i] =
          one ? uint16_t(es ? ((k + 15) << 10) | mant : 0)
              : uint16_t(es ? (cls << 13) | ((k - cls * kClass) << 10) | mant : 0xffff);
    }
    __syncwarp();
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
    for (int at = 0; at < NR; at += 16 * CH) {
      if (at >= n) break;
      if (at > 0) fetch(at);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (at + 16 * c >= n) break;
        uint32_t h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(&weight[warp][at + 16 * c + 2 * t + 8 * q]);
          h[q] = x;  // with a single class all columns are alike
          if (!one) {  // column gq takes class gq
            const uint32_t lo = x & 0xffffu, hi = x >> 16;
            h[q] = (lo != 0xffffu && int(lo >> 13) == gq ? (lo & 0x1fffu) + (15u << 10) : 0u) |
                   (hi != 0xffffu && int(hi >> 13) == gq ? ((hi & 0x1fffu) + (15u << 10)) << 16 : 0u);
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int hh = 0; hh < (VB < 4 ? 1 : 2); ++hh) {
            const uint32_t sel = hh ? 0x7632 : 0x5410;
            const uint32_t a = __byte_perm(v[c][0][w], v[c][1][w], sel);
            const uint32_t d = __byte_perm(v[c][2][w], v[c][3][w], sel);
            if constexpr (BITS == 4) {
              mma16816(acc[4 * w + 2 * hh], a & 0x000f000fu, a & 0x00f000f0u, d & 0x000f000fu,
                       d & 0x00f000f0u, h[0], h[1]);
              const uint32_t e = a >> 8, f = d >> 8;
              mma16816(acc[4 * w + 2 * hh + 1], e & 0x000f000fu, e & 0x00f000f0u, f & 0x000f000fu,
                       f & 0x00f000f0u, h[0], h[1]);
            } else {
              mma16816(acc[2 * w + hh], a & 0x00ff00ffu, (a >> 8) & 0x00ff00ffu, d & 0x00ff00ffu,
                       (d >> 8) & 0x00ff00ffu, h[0], h[1]);
            }
          }
      }
    }
    __syncwarp();  // the weights have been read
    // column c counts 2^(se - 127 + c kClass + 24), upper nibbles 16 times as much
    const double mt = scaled(msum, me - 134);
    double* const o = out + gq * (D / 8);
    if (one) {  // every column has the sums: the four lanes of a row group share the elements
      const int e0 = se - 103, up = BITS == 4 ? 4 : 0;
#pragma unroll
      for (int j = 0; j < (MT + 3) / 4; ++j) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int i = 4 * j; i < (4 * j + 4 < MT ? 4 * j + 4 : MT); ++i)
          if (i % 4 == t) x = acc[i][0], y = acc[i][2];
        if (4 * j + t < MT)
          *reinterpret_cast<double2*>(o + 2 * (4 * j + t)) =
              make_double2(widened(x, e0) + mt, widened(y, e0 - up) + mt);
      }
    } else {
      // whole multiples of 2^(se - 134), the columns' together
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        int64_t v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float unit = BITS == 4 && h ? 0x1p27f : 0x1p31f;
          const int sh = 2 * t * kClass;
          v[h] = sh > kSpread ? 0 : int64_t(__float2int_rn(acc[i][2 * h] * unit)) << sh;
          if (sh + kClass <= kSpread)
            v[h] += int64_t(__float2int_rn(acc[i][2 * h + 1] * unit)) << (sh + kClass);
          v[h] += __shfl_xor_sync(0xffffffffu, v[h], 1);
          v[h] += __shfl_xor_sync(0xffffffffu, v[h], 2);
        }
        if (i % 4 == t) {  // the lanes share the elements
          *reinterpret_cast<double2*>(o + 2 * i) =
              make_double2(scaled(v[0], se - 134) + mt, scaled(v[1], se - 134) + mt);
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

bool al32(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

template <class T, int BITS, int LPR>
void write_rows(const CacheParams& p, const void* K, const void* V, cudaStream_t st) {
  constexpr int RPW = 32 / LPR, UN = 4;
  const T *k = static_cast<const T*>(K), *v = static_cast<const T*>(V);
  const bool wide = al32(K) && al32(V) && p.ks % 8 == 0 && p.vs % 8 == 0;
  // few rows: a warp for each RPW of them
  const bool few = int64_t(p.g.Nq) * p.g.Hkv < int64_t(sm_count()) * 64 * RPW;
  const int64_t tok = few ? RPW : RPW * UN;
  const int64_t warps = (p.g.Nq + tok - 1) / tok * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  if (few) cache_write_kernel<T, BITS, LPR, 1><<<grid, kRowThreads, 0, st>>>(p, k, v, wide);
  else cache_write_kernel<T, BITS, LPR, UN><<<grid, kRowThreads, 0, st>>>(p, k, v, wide);
}

template <class T, int BITS, int LPR>
void read_rows(const CacheParams& p, const int32_t* since, void* K, void* V, cudaStream_t st) {
  constexpr int RPW = 32 / LPR, UN = 4;
  const bool few = int64_t(p.g.Nq) * p.g.Hkv < int64_t(sm_count()) * 64 * RPW;
  const int64_t tok = few ? RPW : RPW * UN;
  const int64_t warps = (p.g.Nq + tok - 1) / tok * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
  const bool wide = al32(K) && al32(V);
  if (few) cache_read_kernel<T, BITS, LPR, 1><<<grid, kRowThreads, 0, st>>>(p, since, k, v, wide);
  else cache_read_kernel<T, BITS, LPR, UN><<<grid, kRowThreads, 0, st>>>(p, since, k, v, wide);
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
  int lz = 0;
  while (since && lz < 6 && (int64_t(p.g.S) * p.g.Hkv << lz) < int64_t(sm_count()) * 32 &&
         int64_t(p.g.block) << lz < p.g.Nk)
    ++lz;
  const int64_t warps = (since ? int64_t(p.g.S) << lz : int64_t(p.g.B)) * p.g.Hkv;
  const unsigned grid = unsigned((warps + 7) / 8);
  by_layout(p, [&](auto bits, auto lpr) {
    if (p.g.block <= 32)
      cache_sums_kernel<bits(), lpr() * 8, 32><<<grid, kRowThreads, 0, st>>>(p, since, sums, lz);
    else if (p.g.block <= 64)
      cache_sums_kernel<bits(), lpr() * 8, 64><<<grid, kRowThreads, 0, st>>>(p, since, sums, lz);
    else
      cache_sums_kernel<bits(), lpr() * 8, 128><<<grid, kRowThreads, 0, st>>>(p, since, sums, lz);
  });
  return launched("gattn_cache_sums");
}

}  // namespace gattn
