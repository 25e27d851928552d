// norm.cu -- the step between two blocks of a transformer layer, fused:
//   u = norm(x; w_post, b_post)        (or u = x)
//   h = res + alpha * gate * u
//   y = norm(h; w_pre, b_pre)          (optional)
// and its backward.  norm is x / rms(x) * w + b or (x - mean) / deviation * w + b.
//
// Both directions are bound by HBM: about 60 flops per element against 4 to
// 11 tensor elements moved.  Each row is read once, kept in registers as fp32
// through both norms, and written once; means, variances, h (before its one
// rounding) and every column sum are fp32.  Variances are sums of squared
// deviations from the mean (two passes over registers, not
// over memory).  The backward forms h
// again from res, x and gate, which costs no traffic over reading h and keeps
// its rounding out of the normalised row (for rows whose mean is large against
// their deviation that rounding would be as large as the row).
//
// A row belongs to W warps; a thread holds E of its elements as 16-byte
// vectors (single elements when a row is no multiple of 16 bytes).  As many CTAs
// as fit run, and each walks its rows; a thread copies its own elements of
// the next rows into shared memory with cp.async, one or two rows ahead -- it
// reads back only what it copied, so the ring needs no barrier, and the bytes
// in flight do not cost registers (80 to 100 KB an SM up to 1,024 columns; the
// backward of longer rows 40 to 80 KB, none beyond 8,192, whose rows are read
// where they are used).  Arithmetic is on pairs
// (fma.rn.f32x2): unpaired, the forward issues 30 instructions an element and
// is bound by them.  Up to 1,024 elements the forward gives a row to one warp
// and needs no block barrier.  The backward carries five fp32 column sums per
// element (dw, db of both norms and the channel gate) over all rows of its
// CTA and keeps its columns' weights in registers; the CTAs' sums meet in a
// second small kernel, in CTA order, so results do not vary from run to run.
// (From 4,097 columns on these sums do not fit its registers: 0.5 to 0.7 KB a
// thread spilled, beyond 8,192 2 to 2.7 KB.)
//
// Measured: 8,192 x 4,096 bf16 forward 52 us (5.1 TB/s); 131,072 x 1,024 bf16 with
// biases and a gate per node 229 us forward (5.9 TB/s) and 394 + 6 us backward (5.4);
// 20,011 x 515 fp32, whose rows are no multiple of 16 bytes, 43 us (3.8) and 58 + 6
// (4.3): single-element copies need four times the instructions; 16 rows of
// 1,024: 3.5 us.
#include <algorithm>

#include "attn_launch.cuh"
#include "attn_pipe.cuh"
#include "block.cuh"

namespace gattn {

namespace {

constexpr int kGateNone = GATTN_GATE_NONE, kGateChannel = GATTN_GATE_CHANNEL,
              kGateToken = GATTN_GATE_TOKEN;
constexpr int kMaxF = 16384;
constexpr int kSums = 5;  // dw_post, db_post, dw_pre, db_pre, dgate (channel)

struct NormParams {
  int64_t N;
  int F;
  float alpha, eps, inv_f;
  int gate_mode;
  const void *res, *x, *gate, *dh, *dy;
  const float *w_post, *b_post, *w_pre, *b_pre;
  void *h, *y, *dres, *dx, *dgate;
  float4* stats;       // [N] (mean, 1/dev) of x, then of h
  const float4* cstats;
  float* part;         // backward: [slots][kSums][F]
  int want;            // bit s: column sum s is wanted
};

// V consecutive elements of a row (16 bytes, or one element) as fp32.
template <class T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
  using Raw = float4;
  __device__ static Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ static void get(const Raw& r, float* f) { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
  __device__ static Raw put(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  __device__ static Raw zero() { return make_uint4(0, 0, 0, 0); }
  __device__ static void get(const Raw& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static Raw put(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float, 1> {
  using Raw = float;
  __device__ static Raw zero() { return 0.f; }
  __device__ static void get(const Raw& r, float* f) { f[0] = r; }
  __device__ static Raw put(const float* f) { return f[0]; }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  __device__ static Raw zero() { return __float2bfloat16(0.f); }
  __device__ static void get(const Raw& r, float* f) { f[0] = __bfloat162float(r); }
  __device__ static Raw put(const float* f) { return __float2bfloat16(f[0]); }
};

// Sums of K values over the W warps of a row.  Warps of one row are a whole
// CTA when W > 1; `turn` alternates the slots so that one barrier per sum is
// enough (a slot is written again only after the next sum's barrier).
template <int W, int K>
__device__ __forceinline__ void row_sums(float* v, float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (W > 1) {
    float* slot = red + turn * W * 2;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) slot[warp * 2 + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += slot[w * 2 + k];
      v[k] = s;
    }
    turn ^= 1;
  }
}

template <class T, int V, int E, int W>
struct Row {
  static constexpr int NV = E / V;
  using R = typename Vec<T, V>::Raw;
  // column of this thread's vector n, and whether the row has it
  __device__ static int col(int n, int t) { return (n * W * 32 + t) * V; }
  __device__ static void load(R* r, const void* base, int64_t row, int F, int t) {
    const T* p = static_cast<const T*>(base) + row * F;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = col(n, t);
      r[n] = c < F ? *reinterpret_cast<const R*>(p + c) : Vec<T, V>::zero();
    }
  }
  __device__ static void store(void* base, int64_t row, int F, int t, const float* f) {
    T* p = static_cast<T*>(base) + row * F;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = col(n, t);
      if (c < F) *reinterpret_cast<R*>(p + c) = Vec<T, V>::put(f + n * V);
    }
  }
  // fp32 channel vector (rows of V elements at column c); `none` where absent
  __device__ static void channel(const float* w, int n, int F, int t, float none, float* f) {
    const int c = col(n, t);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = none;
    if (w && c < F) {
      if constexpr (V == 1) {
        f[0] = w[c];
      } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const float4 a = reinterpret_cast<const float4*>(w + c)[q];
          f[4 * q] = a.x; f[4 * q + 1] = a.y; f[4 * q + 2] = a.z; f[4 * q + 3] = a.w;
        }
      }
    }
  }
};

__device__ __forceinline__ float2 pair(const float* f, int i) {
  return make_float2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void put_pair(float* f, int i, float2 v) {
  f[2 * i] = v.x;
  f[2 * i + 1] = v.y;
}

// zeros past the row's end (`whole`: the row fills its threads)
template <class T, int V, int E, int W>
__device__ __forceinline__ void clip(float* f, int F, int t, bool whole) {
  if (whole) return;
#pragma unroll
  for (int n = 0; n < E / V; ++n)
    if (Row<T, V, E, W>::col(n, t) >= F)
#pragma unroll
      for (int e = 0; e < V; ++e) f[n * V + e] = 0.f;
}

// f becomes (f - mean) / deviation (f / root mean square when LN is false),
// with zeros past the row's end; returns (mean, 1 / deviation)
template <class T, int V, int E, int W, bool LN>
__device__ __forceinline__ float2 normalise(float* f, const NormParams& p, int t, bool whole,
                                            float* red, int& turn) {
  float mean = 0.f;
  if constexpr (LN) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) s2 = f2add(s2, pair(f, i));
    float s[1] = {s2.x + s2.y};
    row_sums<W, 1>(s, red, turn);
    mean = s[0] * p.inv_f;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) put_pair(f, i, f2add(pair(f, i), f2s(-mean)));
    clip<T, V, E, W>(f, p.F, t, whole);
  }
  float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) q2 = f2fma(pair(f, i), pair(f, i), q2);
  float q[1] = {q2.x + q2.y};
  row_sums<W, 1>(q, red, turn);
  const float r = rsqrtf(q[0] * p.inv_f + p.eps);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) put_pair(f, i, f2mul(pair(f, i), f2s(r)));
  return make_float2(mean, r);
}

// the same from statistics that the forward kept
template <class T, int V, int E, int W>
__device__ __forceinline__ void renormalise(float* f, float mean, float r, int F, int t,
                                            bool whole) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) put_pair(f, i, f2mul(f2add(pair(f, i), f2s(-mean)), f2s(r)));
  clip<T, V, E, W>(f, F, t, whole);
}

// A thread's own elements of NT tensors' rows, kStages rows deep in shared
// memory: three or two rows, whatever fits CTAS times on an SM; rows too long
// for two are read from global memory where they are used (kStages 0).
// Elements past the row's end are zeros, written once.
template <class T, int V, int E, int W, int NT, int CTAS, bool DIRECT = false>
struct Ring {
  using RW = Row<T, V, E, W>;
  using R = typename RW::R;
  static constexpr bool kAsync = V * sizeof(T) >= 4;  // cp.async moves 4, 8 or 16 bytes
  static constexpr int kThreads = W == 1 ? 128 : W * 32;
  static constexpr int kTensor = kThreads * RW::NV * int(sizeof(R));
  static constexpr int kRoom = 200 * 1024 / CTAS;
  static constexpr int kStages = DIRECT                        ? 0
                                 : 3 * NT * kTensor <= kRoom ? 3
                                 : 2 * NT * kTensor <= kRoom ? 2
                                                             : 0;
  static constexpr int kBytes = kStages * NT * kTensor;
  uint8_t* base;
  __device__ R* at(int stage, int tensor, int n) const {
    return reinterpret_cast<R*>(base + (stage * NT + tensor) * kTensor) + n * kThreads + threadIdx.x;
  }
  __device__ void clear(int F, int t) {
    for (int s = 0; s < kStages; ++s)
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int n = 0; n < RW::NV; ++n)
          if (RW::col(n, t) >= F) *at(s, k, n) = Vec<T, V>::zero();
  }
  __device__ void fetch(int stage, int tensor, const void* src, int64_t row, int F, int t) {
    const T* p = static_cast<const T*>(src) + row * F;
#pragma unroll
    for (int n = 0; n < RW::NV; ++n) {
      const int c = RW::col(n, t);
      if (c >= F) continue;
      if constexpr (!kAsync) *at(stage, tensor, n) = *reinterpret_cast<const R*>(p + c);
      else if constexpr (sizeof(R) == 16) cp_async16(at(stage, tensor, n), p + c);
      else cp_async4(at(stage, tensor, n), p + c);
    }
  }
  // the elements of `row`, the k-th that this CTA walks (vector n, or all)
  __device__ void get1(int k, int tensor, int n, const void* src, int64_t row, int F, int t,
                       float* f) const {
    if constexpr (kStages == 0) {
      const int c = RW::col(n, t);
      const T* p = static_cast<const T*>(src) + row * F;
      Vec<T, V>::get(c < F ? *reinterpret_cast<const R*>(p + c) : Vec<T, V>::zero(), f);
    } else {
      Vec<T, V>::get(*at(k % kStages, tensor, n), f);
    }
  }
  __device__ void get(int k, int tensor, const void* src, int64_t row, int F, int t,
                      float* f) const {
#pragma unroll
    for (int n = 0; n < RW::NV; ++n) get1(k, tensor, n, src, row, F, t, f + n * V);
  }
  __device__ void wait() const {
    if constexpr (kStages > 0) cp_async_wait<kStages - 2>();
  }
};

template <class T, int V, int E, int W>
__device__ __forceinline__ void channels(const float* w, int F, int t, float none, float* f) {
#pragma unroll
  for (int n = 0; n < E / V; ++n) Row<T, V, E, W>::channel(w, n, F, t, none, f + n * V);
}

// CTAs per SM: registers a thread of about 64 (E = 8), 80 (16) and 128 forward,
// 128 backward
template <int E, int W>
constexpr int fwd_ctas() {
  const int threads = W == 1 ? 128 : W * 32, most = E <= 8 ? 1024 : E <= 16 ? 768 : 512;
  return most < threads ? 1 : most / threads;
}
template <int W>
constexpr int bwd_ctas() {
  return W <= 4 ? 4 : 1;
}

template <class T, int V, int E, int W, bool LN>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32, fwd_ctas<E, W>())
    norm_fwd_kernel(const NormParams p) {
  using RW = Row<T, V, E, W>;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[W > 1 ? 4 * W : 1];
  // single bf16 elements are too small for cp.async: many short-lived CTAs
  // read them directly
  using Rg = Ring<T, V, E, W, 3, fwd_ctas<E, W>(), V * sizeof(T) < 4>;
  Rg ring{ring_mem};
  int turn = 0;
  const int t = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t slot = W == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = W == 1 ? int64_t(gridDim.x) * 4 : gridDim.x;
  const bool token = p.gate_mode == kGateToken, whole = p.F == E * W * 32;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.N) {
      ring.fetch(stage, 0, p.res, row, p.F, t);
      if (p.x) ring.fetch(stage, 1, p.x, row, p.F, t);
      if (p.x && token) ring.fetch(stage, 2, p.gate, row, p.F, t);
    }
    cp_async_commit();
  };
  if (!whole) ring.clear(p.F, t);
  for (int s = 0; s < Rg::kStages - 1; ++s) fetch(slot + s * step, s);
  int k = 0;
  for (int64_t row = slot; row < p.N; row += step, ++k) {
    ring.wait();
    // (the stage that is refilled was read a row ago)
    if constexpr (Rg::kStages > 0)
      fetch(row + (Rg::kStages - 1) * step, (k + Rg::kStages - 1) % Rg::kStages);
    float h[E];
    if constexpr (Rg::kStages == 0) ring.get(k, 0, p.res, row, p.F, t, h);
    if (p.x) {
      float u[E];
      ring.get(k, 1, p.x, row, p.F, t, u);
      if (p.w_post) {
        const float2 s = normalise<T, V, E, W, LN>(u, p, t, whole, red, turn);
        if (t == 0) reinterpret_cast<float2*>(p.stats + row)[0] = s;
      }
      if constexpr (Rg::kStages > 0) ring.get(k, 0, p.res, row, p.F, t, h);
#pragma unroll
      for (int n = 0; n < RW::NV; ++n) {
        float w[V], b[V], g[V];
        if (token)
          ring.get1(k, 2, n, p.gate, row, p.F, t, g);
        else
          RW::channel(p.gate_mode == kGateChannel ? static_cast<const float*>(p.gate) : nullptr, n,
                      p.F, t, 1.f, g);
        if (p.w_post) {
          RW::channel(p.w_post, n, p.F, t, 0.f, w);
          RW::channel(p.b_post, n, p.F, t, 0.f, b);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int i = n * V + e;
          if (p.w_post) u[i] = fmaf(u[i], w[e], b[e]);
          h[i] = fmaf(g[e] * p.alpha, u[i], h[i]);
        }
      }
      RW::store(p.h, row, p.F, t, h);
    } else if constexpr (Rg::kStages > 0) {
      ring.get(k, 0, p.res, row, p.F, t, h);
    }
    if (p.w_pre) {  // on h as it stands in fp32, not as rounded for the store
      const float2 s = normalise<T, V, E, W, LN>(h, p, t, whole, red, turn);
      if (t == 0) reinterpret_cast<float2*>(p.stats + row)[1] = s;
#pragma unroll
      for (int n = 0; n < RW::NV; ++n) {
        float w[V], b[V];
        RW::channel(p.w_pre, n, p.F, t, 0.f, w);
        RW::channel(p.b_pre, n, p.F, t, 0.f, b);
#pragma unroll
        for (int e = 0; e < V; ++e) h[n * V + e] = fmaf(h[n * V + e], w[e], b[e]);
      }
      RW::store(p.y, row, p.F, t, h);
    }
  }
  cp_async_wait<0>();
}

// dx of a norm: g = dy * w, xh the normalised row, r = 1 / deviation
//   dx = r (g - xh mean(g xh) - [LN] mean(g));  absent columns hold g = xh = 0
template <int E, int W, bool LN>
__device__ __forceinline__ void norm_dx(float* g, const float* xh, float r, float inv_f, float* red,
                                        int& turn) {
  float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    a = f2fma(pair(g, i), pair(xh, i), a);
    if (LN) b = f2add(b, pair(g, i));
  }
  float s[2] = {a.x + a.y, b.x + b.y};
  row_sums<W, LN ? 2 : 1>(s, red, turn);
  const float2 c1 = f2s(-s[0] * inv_f), c2 = f2s(LN ? -s[1] * inv_f : 0.f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    float2 v = f2fma(pair(xh, i), c1, pair(g, i));
    if (LN) v = f2add(v, c2);
    put_pair(g, i, f2mul(v, f2s(r)));
  }
}

template <class T, int V, int E, int W, bool LN>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32, bwd_ctas<W>())
    norm_bwd_kernel(const NormParams p) {
  using RW = Row<T, V, E, W>;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[W > 1 ? 4 * W : 1];
  using Rg = Ring<T, V, E, W, 5, bwd_ctas<W>()>;
  Rg ring{ring_mem};
  int turn = 0;
  const int t = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t slot = W == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = W == 1 ? int64_t(gridDim.x) * 4 : gridDim.x;
  const bool has_x = p.x != nullptr, token = p.gate_mode == kGateToken;
  const bool whole = p.F == E * W * 32;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.N) {
      if (p.w_pre) {
        ring.fetch(stage, 0, p.res, row, p.F, t);
        ring.fetch(stage, 1, p.dy, row, p.F, t);
      }
      if (p.dh) ring.fetch(stage, 2, p.dh, row, p.F, t);
      if (has_x) {
        ring.fetch(stage, 3, p.x, row, p.F, t);
        if (token) ring.fetch(stage, 4, p.gate, row, p.F, t);
      }
    }
    cp_async_commit();
  };
  if (!whole) ring.clear(p.F, t);
  for (int s = 0; s < Rg::kStages - 1; ++s) fetch(slot + s * step, s);
  float acc[kSums][E];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
  constexpr bool KEEP = E <= 8;  // weights stay in registers
  float wa[E], ba[E], wb[E], gc[E];
  auto weights = [&]() {
    channels<T, V, E, W>(p.w_post, p.F, t, 0.f, wa);
    channels<T, V, E, W>(p.b_post, p.F, t, 0.f, ba);
    channels<T, V, E, W>(p.w_pre, p.F, t, 0.f, wb);
    channels<T, V, E, W>(p.gate_mode == kGateChannel ? static_cast<const float*>(p.gate) : nullptr,
                         p.F, t, 1.f, gc);
  };
  if (KEEP) weights();
  float4 next = slot < p.N ? p.cstats[slot] : make_float4(0.f, 0.f, 0.f, 0.f);
  int k = 0;
  for (int64_t row = slot; row < p.N; row += step, ++k) {
    const float4 s = next;
    if (row + step < p.N) next = p.cstats[row + step];
    ring.wait();
    if (!KEEP) weights();
    // x becomes its normalised row; hh that of h, formed again as the forward did
    // (the stage that is refilled was read a row ago)
    if constexpr (Rg::kStages > 0)
      fetch(row + (Rg::kStages - 1) * step, (k + Rg::kStages - 1) % Rg::kStages);
    float d[E], x[E], g[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (has_x) ring.get(k, 3, p.x, row, p.F, t, x);
    if (token) {
      ring.get(k, 4, p.gate, row, p.F, t, g);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = gc[e];
    }
    if (p.w_post) renormalise<T, V, E, W>(x, s.x, s.y, p.F, t, whole);
    if (p.w_pre) {
      float hh[E], gy[E];
      ring.get(k, 0, p.res, row, p.F, t, hh);
      if (has_x) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float2 u = p.w_post ? f2fma(pair(x, i), pair(wa, i), pair(ba, i)) : pair(x, i);
          put_pair(hh, i, f2fma(f2mul(pair(g, i), f2s(p.alpha)), u, pair(hh, i)));
        }
      }
      renormalise<T, V, E, W>(hh, s.z, s.w, p.F, t, whole);
      ring.get(k, 1, p.dy, row, p.F, t, gy);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        put_pair(acc[2], i, f2fma(pair(gy, i), pair(hh, i), pair(acc[2], i)));
        put_pair(acc[3], i, f2add(pair(acc[3], i), pair(gy, i)));
        put_pair(gy, i, f2mul(pair(gy, i), pair(wb, i)));
      }
      norm_dx<E, W, LN>(gy, hh, s.w, p.inv_f, red, turn);
      if (p.dh) {
        ring.get(k, 2, p.dh, row, p.F, t, d);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) put_pair(d, i, f2add(pair(d, i), pair(gy, i)));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = gy[e];
      }
    } else {
      ring.get(k, 2, p.dh, row, p.F, t, d);
    }
    if (p.dres) RW::store(p.dres, row, p.F, t, d);
    if (!has_x) continue;
    // d = gradient of h; du = alpha gate d
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 ad = f2mul(pair(d, i), f2s(p.alpha));
      const float2 u = p.w_post ? f2fma(pair(x, i), pair(wa, i), pair(ba, i)) : pair(x, i);
      const float2 du = f2mul(ad, pair(g, i));
      put_pair(g, i, f2mul(ad, u));  // the gate's gradient
      put_pair(acc[4], i, f2add(pair(acc[4], i), pair(g, i)));
      put_pair(acc[0], i, f2fma(du, pair(x, i), pair(acc[0], i)));
      put_pair(acc[1], i, f2add(pair(acc[1], i), du));
      put_pair(d, i, p.w_post ? f2mul(du, pair(wa, i)) : du);
    }
    if (token && p.dgate) RW::store(p.dgate, row, p.F, t, g);
    if (p.w_post) norm_dx<E, W, LN>(d, x, s.y, p.inv_f, red, turn);
    if (p.dx) RW::store(p.dx, row, p.F, t, d);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int k = 0; k < kSums; ++k)
    if ((p.want >> k) & 1) {
      float* o = p.part + (slot * kSums + k) * p.F;
#pragma unroll
      for (int n = 0; n < RW::NV; ++n) {
        const int c = RW::col(n, t);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c < p.F) o[c + e] = acc[k][n * V + e];
      }
    }
}

// Column sums over the slots, in slot order within each of 32 fixed strands.
struct NormOut {
  float* o[kSums];
};
__global__ void __launch_bounds__(1024) norm_cols_kernel(const float* part, int slots, int F,
                                                         NormOut out) {
  __shared__ float sh[32][33];
  const int k = blockIdx.y, lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
  if (!out.o[k]) return;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < F) {
#pragma unroll 8
    for (int i = strand; i < slots; i += 32) s += part[(int64_t(i) * kSums + k) * F + c];
  }
  sh[strand][lane] = s;
  __syncthreads();
  // warp w adds up column w of the block's 32
  float v = sh[lane][strand];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + strand < F) out.o[k][blockIdx.x * 32 + strand] = v;
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------
bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gattn_status fail(gattn_status s, const char* msg) {
  set_error("gattn_norm: %s", msg);
  return s;
}

gattn_status check_desc(const gattn_norm_desc* d) {
  if (!d) return fail(GATTN_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != GATTN_F32 && d->dtype != GATTN_BF16)
    return fail(GATTN_ERR_INVALID_ARG, "unknown dtype");
  if (d->kind != GATTN_NORM_RMS && d->kind != GATTN_NORM_LAYER)
    return fail(GATTN_ERR_INVALID_ARG, "unknown kind");
  if (d->gate != kGateNone && d->gate != kGateChannel && d->gate != kGateToken)
    return fail(GATTN_ERR_INVALID_ARG, "unknown gate mode");
  if (d->N < 0 || d->F <= 0 || d->N > INT32_MAX)
    return fail(GATTN_ERR_INVALID_ARG, "need 0 <= N < 2^31 and F > 0");
  if (d->F > kMaxF) return fail(GATTN_ERR_UNSUPPORTED, "F must be at most 16384");
  if ((d->b_post && !d->w_post) || (d->b_pre && !d->w_pre))
    return fail(GATTN_ERR_INVALID_ARG, "a bias needs its weight");
  if (!al(d->w_post, 16) || !al(d->b_post, 16) || !al(d->w_pre, 16) || !al(d->b_pre, 16))
    return fail(GATTN_ERR_INVALID_ARG, "weights and biases must be 16-byte aligned");
  return GATTN_OK;
}

NormParams params(const gattn_norm_desc* d) {
  NormParams p{};
  p.N = d->N;
  p.F = d->F;
  p.alpha = d->alpha;
  p.eps = d->eps;
  p.inv_f = 1.f / float(d->F);
  p.gate_mode = d->gate;
  p.w_post = d->w_post;
  p.b_post = d->b_post;
  p.w_pre = d->w_pre;
  p.b_pre = d->b_pre;
  return p;
}

// Whole 16-byte vectors fit when the row size is a multiple of 16 bytes.
bool vectors(const gattn_norm_desc* d) {
  return (int64_t(d->F) * (d->dtype == GATTN_F32 ? 4 : 2)) % 16 == 0;
}

gattn_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s launch failed: %s", what, cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  return GATTN_OK;
}

template <class K>
void launch_ring(K kern, unsigned grid, int threads, int bytes, const NormParams& p,
                 cudaStream_t st) {
  if (bytes > 40 * 1024)  // static shared memory counts towards the 48 KB too
    cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  kern<<<grid, threads, bytes, st>>>(p);
}

template <class T, int V, int E, int W, bool LN>
void fwd_go(const NormParams& p, cudaStream_t st) {
  constexpr int CTAS = fwd_ctas<E, W>();
  const int64_t ctas = W == 1 ? (p.N + 3) / 4 : p.N;
  using Rg = Ring<T, V, E, W, 3, CTAS, V * sizeof(T) < 4>;
  const unsigned grid = unsigned(
      Rg::kStages == 0 ? ctas : std::min<int64_t>(ctas, int64_t(CTAS) * sm_count()));
  launch_ring(norm_fwd_kernel<T, V, E, W, LN>, grid, W == 1 ? 128 : W * 32, Rg::kBytes, p, st);
}

// Elements a thread and warps a row: the fewest elements that cover the row (in
// steps, so that few kernels are compiled); one warp a row up to 1,024 (no
// barriers), from there 16 elements a thread.  Rows in single elements take
// four warps from 257 on, because 24 or 32 copies of 4 bytes a lane are slower
// than the barriers (20,011 x 515 fp32: 84 us with one warp, 43 with four).
template <class T, int V, bool LN>
void fwd_launch(const NormParams& p, cudaStream_t st) {
  if (p.F <= 256) fwd_go<T, V, 8, 1, LN>(p, st);
  else if (p.F <= 512) fwd_go<T, V, V == 1 ? 4 : 16, V == 1 ? 4 : 1, LN>(p, st);
  else if (p.F <= 768) fwd_go<T, V, V == 1 ? 6 : 24, V == 1 ? 4 : 1, LN>(p, st);
  else if (p.F <= 1024) fwd_go<T, V, V == 1 ? 8 : 32, V == 1 ? 4 : 1, LN>(p, st);
  else if (p.F <= 2048) fwd_go<T, V, 16, 4, LN>(p, st);
  else if (p.F <= 4096) fwd_go<T, V, 16, 8, LN>(p, st);
  else if (p.F <= 8192) fwd_go<T, V, 16, 16, LN>(p, st);
  else fwd_go<T, V, 32, 16, LN>(p, st);
}

template <class T, int V>
void fwd_kind(const NormParams& p, bool ln, cudaStream_t st) {
  if (ln) fwd_launch<T, V, true>(p, st);
  else fwd_launch<T, V, false>(p, st);
}

// Shape of the backward: warps per row and rows in flight.
struct BwdShape {
  int warps, slots;  // slots: partial column sums (one per row in flight)
  unsigned grid;
};
BwdShape bwd_shape(const gattn_norm_desc* d) {
  BwdShape s{};
  s.warps = d->F <= 256 ? 1 : d->F <= 1024 ? 4 : 16;
  const int64_t per_sm = s.warps <= 4 ? 4 : 1;  // bwd_ctas
  const int64_t rows = s.warps == 1 ? (d->N + 3) / 4 : d->N;
  s.grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(rows, per_sm * sm_count())));
  s.slots = int(s.grid) * (s.warps == 1 ? 4 : 1);
  return s;
}

template <class T, int V, int E, int W, bool LN>
void bwd_go(const NormParams& p, const BwdShape& s, cudaStream_t st) {
  launch_ring(norm_bwd_kernel<T, V, E, W, LN>, s.grid, W == 1 ? 128 : W * 32,
              Ring<T, V, E, W, 5, bwd_ctas<W>()>::kBytes, p, st);
}

template <class T, int V, bool LN>
void bwd_launch(const NormParams& p, const BwdShape& s, cudaStream_t st) {
  if (s.warps == 1) bwd_go<T, V, 8, 1, LN>(p, s, st);
  else if (p.F <= 512 && V <= 4) bwd_go<T, V, V <= 4 ? 4 : 8, 4, LN>(p, s, st);
  else if (p.F <= 768 && V == 1) bwd_go<T, V, V == 1 ? 6 : 8, 4, LN>(p, s, st);
  else if (s.warps == 4) bwd_go<T, V, 8, 4, LN>(p, s, st);
  else if (p.F <= 4096) bwd_go<T, V, 8, 16, LN>(p, s, st);
  else if (p.F <= 8192) bwd_go<T, V, 16, 16, LN>(p, s, st);
  else bwd_go<T, V, 32, 16, LN>(p, s, st);
}

template <class T, int V>
void bwd_kind(const NormParams& p, const BwdShape& s, bool ln, cudaStream_t st) {
  if (ln) bwd_launch<T, V, true>(p, s, st);
  else bwd_launch<T, V, false>(p, s, st);
}

}  // namespace

}  // namespace gattn

using namespace gattn;

extern "C" {

gattn_status gattn_norm_fwd(const gattn_norm_desc* d, const void* res, const void* x,
                            const void* gate, void* h, void* y, float* stats,
                            gattn_stream_t stream) {
  gattn_status s = check_desc(d);
  if (s != GATTN_OK) return s;
  if (d->N == 0) return GATTN_OK;
  if (!x && (d->w_post || d->gate != kGateNone || gate))
    return fail(GATTN_ERR_INVALID_ARG, "w_post and gate need x");
  if (!x && !d->w_pre) return fail(GATTN_ERR_INVALID_ARG, "nothing to compute: give x or w_pre");
  if (!res || !al(res, 16) || !al(x, 16) || (x && (!h || !al(h, 16))) ||
      (d->w_pre && (!y || !al(y, 16))) || !stats || !al(stats, 16) ||
      (d->gate != kGateNone && (!gate || !al(gate, 16))))
    return fail(GATTN_ERR_INVALID_ARG,
                "res, x, gate, h, y and stats must be 16-byte aligned device pointers");
  NormParams p = params(d);
  p.res = res;
  p.x = x;
  p.gate = gate;
  p.h = h;
  p.y = y;
  p.stats = reinterpret_cast<float4*>(stats);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool ln = d->kind == GATTN_NORM_LAYER;
  if (d->dtype == GATTN_F32) {
    if (vectors(d)) fwd_kind<float, 4>(p, ln, st);
    else fwd_kind<float, 1>(p, ln, st);
  } else {
    if (vectors(d)) fwd_kind<__nv_bfloat16, 8>(p, ln, st);
    else fwd_kind<__nv_bfloat16, 1>(p, ln, st);
  }
  return launched("gattn_norm_fwd");
}

gattn_status gattn_norm_workspace_size(const gattn_norm_desc* d, size_t* bytes) {
  const gattn_status s = check_desc(d);
  if (s != GATTN_OK) return s;
  if (!bytes) return fail(GATTN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = size_t(bwd_shape(d).slots) * kSums * d->F * sizeof(float);
  return GATTN_OK;
}

gattn_status gattn_norm_bwd(const gattn_norm_desc* d, const void* res, const float* stats,
                            const void* dh, const void* dy, const void* x, const void* gate,
                            void* dres, void* dx, void* dgate, float* dw_post, float* db_post,
                            float* dw_pre, float* db_pre, void* workspace, size_t workspace_bytes,
                            gattn_stream_t stream) {
  gattn_status s = check_desc(d);
  if (s != GATTN_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  float* chan = d->gate == kGateChannel ? static_cast<float*>(dgate) : nullptr;
  const NormOut out{{dw_post, db_post, dw_pre, db_pre, chan}};
  if (d->N == 0) {  // sums over no rows
    for (float* o : out.o)
      if (o && cudaMemsetAsync(o, 0, size_t(d->F) * 4, st) != cudaSuccess)
        return fail(GATTN_ERR_CUDA, "cudaMemsetAsync failed");
    return GATTN_OK;
  }
  if (!x && (d->w_post || d->gate != kGateNone || gate || dx || dgate))
    return fail(GATTN_ERR_INVALID_ARG, "w_post, gate, dx and dgate need x");
  if ((!d->w_post && (dw_post || db_post)) || (!d->w_pre && (dw_pre || db_pre || dy)) ||
      (d->gate == kGateNone && dgate))
    return fail(GATTN_ERR_INVALID_ARG, "a gradient is asked for that has no operand");
  if (d->w_pre && !dy) return fail(GATTN_ERR_INVALID_ARG, "dy is NULL");
  if (!dh && !d->w_pre) return fail(GATTN_ERR_INVALID_ARG, "neither dh nor dy is given");
  const BwdShape sh = bwd_shape(d);
  const size_t need = size_t(sh.slots) * kSums * d->F * sizeof(float);
  if ((d->w_pre && (!res || !al(res, 16))) || !stats || !al(stats, 16) || !al(dh, 16) || !al(dy, 16) ||
      !al(x, 16) || (d->gate != kGateNone && (!gate || !al(gate, 16))) || !al(dres, 16) ||
      !al(dx, 16) || !al(dgate, 16) || !al(dw_post, 4) || !al(db_post, 4) || !al(dw_pre, 4) ||
      !al(db_pre, 4))
    return fail(GATTN_ERR_INVALID_ARG, "tensors must be 16-byte aligned device pointers");
  if (!workspace || !al(workspace, 16) || workspace_bytes < need) {
    set_error("gattn_norm_bwd: workspace needs %zu bytes (16-byte aligned), got %zu", need,
              workspace_bytes);
    return GATTN_ERR_INVALID_ARG;
  }
  NormParams p = params(d);
  p.res = res;
  p.cstats = reinterpret_cast<const float4*>(stats);
  p.dh = dh;
  p.dy = dy;
  p.x = x;
  p.gate = gate;
  p.dres = dres;
  p.dx = dx;
  p.dgate = dgate;
  p.part = static_cast<float*>(workspace);
  for (int k = 0; k < kSums; ++k) p.want |= out.o[k] ? 1 << k : 0;
  const bool ln = d->kind == GATTN_NORM_LAYER;
  if (d->dtype == GATTN_F32) {
    if (vectors(d)) bwd_kind<float, 4>(p, sh, ln, st);
    else bwd_kind<float, 1>(p, sh, ln, st);
  } else {
    if (vectors(d)) bwd_kind<__nv_bfloat16, 8>(p, sh, ln, st);
    else bwd_kind<__nv_bfloat16, 1>(p, sh, ln, st);
  }
  if ((s = launched("gattn_norm_bwd")) != GATTN_OK || !p.want) return s;
  norm_cols_kernel<<<dim3((d->F + 31) / 32, kSums), 1024, 0, st>>>(p.part, sh.slots, d->F, out);
  return launched("gattn_norm_bwd (column sums)");
}

}  // extern "C"
