// rotary.cu -- rotary positions of Q and K in one launch, and their frequencies.
//
// An angle is position * frequency modulo a turn.  Frequencies are 64-bit
// fractions of a turn, so the product wraps to the exact fraction with one
// integer multiplication at any position; its top 32 bits are split into the
// quarter and a rest in [-1/8, 1/8) turns that fp32 holds to 2^-28, and sine and
// cosine of the rest are taken in fp32.
//
// The rows are read and written once: the bound is HBM.  A thread owns the two
// 16-byte vectors of a row that turn together (halves), or one (neighbours), and
// walks over heads with the sines that it formed once; with few rows it takes
// fewer heads, so that there are threads enough.
//
// Measured: 32,768 rows of 32 + 8 heads of 128 in bf16 103 us (6.5 TB/s of reads and writes, 0.97 of
// a copy), in fp32 198; 20,013 rows of 8 + 8 heads of 64 in fp32 27 us (5.9 TB/s); 16 rows 3.9 us,
// latency.  The first with a width of 96 119 us, of 10 in halves, whose partners lie on no border, 154, of 10 with neighbours 105.
#include <cmath>

#include "cache.cuh"

namespace gattn {

namespace {

constexpr int kRotThreads = 256;

struct RotParams {
  int N, H, HT, D, R, S;  // HT: heads of Q and K together
  int cph, hg, rpb;       // threads per head, heads side by side, rows per block
  int flat;               // elements of a head from here on move as vectors (D: none)
  bool half;
  float amp, sign;
  const uint64_t* freqs;
  const int32_t *pos, *seq_q, *seq_k, *len_k;
  const char *q, *k;
  char *qo, *ko;
  int64_t qs, ks, qos, kos;  // row strides in elements
};

__device__ __forceinline__ bool position(const RotParams& p, int r, int64_t* at) {
  if (p.pos) {
    *at = p.pos[r];
    return true;
  }
  const SeqRow x = seq_row(p.seq_q, p.S, p.N, r);
  if (x.s < 0) return false;
  int64_t len = p.len_k ? int64_t(p.len_k[x.s]) : x.n;
  if (p.seq_k) {  // the attention cuts lengths to the room
    const int64_t room = max(int64_t(p.seq_k[x.s + 1]) - p.seq_k[x.s], int64_t(0));
    len = p.len_k ? max(min(len, room), int64_t(0)) : room;
  }
  *at = len - x.n + x.i;
  return true;
}

// amp * cos and amp * sin of `at` * freq turns
__device__ __forceinline__ void turn(const RotParams& p, int64_t at, uint64_t freq, float* c,
                                     float* s) {
  const uint32_t t = uint32_t((uint64_t(at) * freq) >> 32);
  const uint32_t q = (t + 0x20000000u) >> 30;  // nearest quarter
  const float x = float(int32_t(t - (q << 30))) * 0x1p-31f;  // half turns in [-1/4, 1/4)
  float sn, cs;
  sincospif(x, &sn, &cs);
  const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
  *c = (q == 1 || q == 2 ? -a : a) * p.amp;
  *s = (q >= 2 ? -b : b) * p.amp * p.sign;
}

template <class T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int V = 4;
  __device__ static void get(uint4 a, float* f) {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
  }
  __device__ static uint4 put(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int V = 8;
  __device__ static void get(uint4 a, float* f) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 put(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Whole vectors.  Thread j of a head has, with halves, vector j of the first half and its partner
// in the second; else vector j alone, whose pairs are neighbours.  What lies behind the
// first R elements is copied.
template <class T, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotParams p) {
  constexpr int V = Pack<T>::V;
  constexpr int NV = HALF ? 2 : 1;  // vectors of a thread and head
  constexpr int NP = V * NV / 2;    // pairs
  constexpr int UN = 8 / NV;        // heads on their way at a time
  const int per_row = p.cph * p.hg;
  const int lr = threadIdx.x / per_row, rem = threadIdx.x - lr * per_row;
  const int64_t row = int64_t(blockIdx.x) * p.rpb + lr;
  if (lr >= p.rpb || row >= p.N) return;
  const int h0 = rem / p.cph, j = rem - h0 * p.cph;
  int64_t at;
  if (!position(p, int(row), &at)) return;
  const T* q = reinterpret_cast<const T*>(p.q) + row * p.qs;
  const T* k = reinterpret_cast<const T*>(p.k) + row * p.ks;
  T* qo = reinterpret_cast<T*>(p.qo) + row * p.qos;
  T* ko = reinterpret_cast<T*>(p.ko) + row * p.kos;
  const auto src = [&](int h) { return h < p.H ? q + h * p.D : k + (h - p.H) * p.D; };
  const auto dst = [&](int h) { return h < p.H ? qo + h * p.D : ko + (h - p.H) * p.D; };
  // pairs of the thread that turn: with halves all or none, else those within R
  const int turning = HALF ? p.R / (2 * V) : 0;
  const int live = HALF ? (j < turning ? NP : 0) : clampi(p.R / 2 - j * NP, 0, NP);
  const bool turns = live > 0;
  const int oa = !HALF || turns ? j * V : p.R + (j - turning) * V;
  const int ob = oa + (HALF && turns ? p.R / 2 : 0);
  float c[NP], s[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
    if (i < live) turn(p, at, p.freqs[j * NP + i], &c[i], &s[i]);
  }
  for (int h = h0; h < p.HT; h += UN * p.hg) {
    uint4 a[UN], b[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (h + u * p.hg < p.HT) {
        const T* x = src(h + u * p.hg);
        a[u] = *reinterpret_cast<const uint4*>(x + oa);
        if (HALF) b[u] = *reinterpret_cast<const uint4*>(x + ob);
      }
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (h + u * p.hg < p.HT) {
        T* z = dst(h + u * p.hg);
        if (!turns) {
          *reinterpret_cast<uint4*>(z + oa) = a[u];
          continue;
        }
        float f[NV * V], o[NV * V];
        Pack<T>::get(a[u], f);
        if (HALF) Pack<T>::get(b[u], f + V * (NV - 1));
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int x = HALF ? i : 2 * i, y = HALF ? i + V : 2 * i + 1;
          const bool on = HALF || i < live;
          o[x] = on ? f[x] * c[i] - f[y] * s[i] : f[x];
          o[y] = on ? f[x] * s[i] + f[y] * c[i] : f[y];
        }
        *reinterpret_cast<uint4*>(z + oa) = Pack<T>::put(o);
        if (HALF) *reinterpret_cast<uint4*>(z + ob) = Pack<T>::put(o + V * (NV - 1));
      }
  }
}

// Any alignment and width.  Thread j of a head turns pair j, copies an element behind the pairs, or,
// from element `flat` on, a whole vector.
template <class T>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotParams p) {
  constexpr int V = Pack<T>::V;
  constexpr int UN = 4;  // heads on their way at a time
  const int64_t n = int64_t(p.N) * p.cph;
  for (int64_t e = int64_t(blockIdx.x) * kRotThreads + threadIdx.x; e < n;
       e += int64_t(gridDim.x) * kRotThreads) {
    const int64_t row = e / p.cph;
    const int j = int(e - row * p.cph);
    int64_t at;
    if (!position(p, int(row), &at)) continue;
    const T* q = reinterpret_cast<const T*>(p.q) + row * p.qs;
    const T* k = reinterpret_cast<const T*>(p.k) + row * p.ks;
    T* qo = reinterpret_cast<T*>(p.qo) + row * p.qos;
    T* ko = reinterpret_cast<T*>(p.ko) + row * p.kos;
    const auto src = [&](int h) { return h < p.H ? q + h * p.D : k + (h - p.H) * p.D; };
    const auto dst = [&](int h) { return h < p.H ? qo + h * p.D : ko + (h - p.H) * p.D; };
    const int singles = p.R / 2 + p.flat - p.R;  // pairs, and elements behind them
    const int step = gridDim.y;
    if (j >= singles) {
      const int o = p.flat + (j - singles) * V;
      for (int h = blockIdx.y; h < p.HT; h += UN * step) {
        uint4 a[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (h + u * step < p.HT) a[u] = *reinterpret_cast<const uint4*>(src(h + u * step) + o);
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (h + u * step < p.HT) *reinterpret_cast<uint4*>(dst(h + u * step) + o) = a[u];
      }
      continue;
    }
    const bool pair = j < p.R / 2;
    const int oa = !pair ? p.R / 2 + j : p.half ? j : 2 * j;
    const int ob = !pair ? oa : p.half ? j + p.R / 2 : 2 * j + 1;
    float c = 1.f, s = 0.f;
    if (pair) turn(p, at, p.freqs[j], &c, &s);
    for (int h = blockIdx.y; h < p.HT; h += UN * step) {
      T a[UN], b[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u)
        if (h + u * step < p.HT) {
          a[u] = src(h + u * step)[oa];
          b[u] = src(h + u * step)[ob];
        }
#pragma unroll
      for (int u = 0; u < UN; ++u)
        if (h + u * step < p.HT) {
          T* z = dst(h + u * step);
          if (!pair) {
            z[oa] = a[u];
            continue;
          }
          const float x = float(a[u]), y = float(b[u]);
          z[oa] = T(x * c - y * s);
          z[ob] = T(x * s + y * c);
        }
    }
  }
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define ROT_REQUIRE(cond, code, ...)           \
  do {                                         \
    if (!(cond)) {                             \
      set_error("gattn_rotary: " __VA_ARGS__); \
      return code;                             \
    }                                          \
  } while (0)

template <class T>
void launch(RotParams& p, bool vectors, bool whole, cudaStream_t st) {
  constexpr int V = Pack<T>::V;
  if (!whole) {
    p.flat = vectors ? (p.R + V - 1) / V * V : p.D;
    p.cph = p.R / 2 + (p.flat - p.R) + (p.D - p.flat) / V;
    const int64_t n = (int64_t(p.N) * p.cph + kRotThreads - 1) / kRotThreads;
    // heads in groups of blocks as long as the rows alone do not fill the GPU eight times
    int heads = 1;
    while (heads < p.HT && heads < 64 && n * heads < int64_t(sm_count()) * 64) heads *= 2;
    rotary_any_kernel<T><<<dim3(unsigned(n < 1 << 20 ? n : 1 << 20), heads), kRotThreads, 0, st>>>(p);
    return;
  }
  p.cph = p.half ? p.R / (2 * V) + (p.D - p.R) / V : p.D / V;
  // heads side by side: the fewest that give every SM about 1,024 threads, since every thread of a
  // row forms the same sines again
  const int64_t want = int64_t(sm_count()) * 1024;
  int hg = 1;
  while (hg < p.HT && 2 * hg * p.cph <= kRotThreads &&
         (int64_t(p.N) * hg * p.cph < want || hg * p.cph < 32))
    hg *= 2;
  p.hg = hg;
  p.rpb = kRotThreads / (p.cph * hg);
  const int64_t blocks = (int64_t(p.N) + p.rpb - 1) / p.rpb;
  if (p.half) rotary_kernel<T, true><<<unsigned(blocks), kRotThreads, 0, st>>>(p);
  else rotary_kernel<T, false><<<unsigned(blocks), kRotThreads, 0, st>>>(p);
}

}  // namespace

}  // namespace gattn

using namespace gattn;

extern "C" {

gattn_status gattn_rotary(const gattn_rotary_desc* d, const void* Q, const void* K, void* Q_out,
                          void* K_out, gattn_stream_t stream) {
  ROT_REQUIRE(d != nullptr, GATTN_ERR_INVALID_ARG, "desc is NULL");
  ROT_REQUIRE(d->dtype == GATTN_F32 || d->dtype == GATTN_BF16, GATTN_ERR_INVALID_ARG,
              "unknown dtype %d", d->dtype);
  ROT_REQUIRE(d->N >= 0 && d->H > 0 && d->Hkv >= 0 && d->D > 0 && d->S >= 0, GATTN_ERR_INVALID_ARG,
              "N, Hkv and S must not be negative, H and D positive (%d, %d, %d, %d, %d)", d->N,
              d->Hkv, d->S, d->H, d->D);
  ROT_REQUIRE(d->D <= 1024 && int64_t(d->H) + d->Hkv <= 65536, GATTN_ERR_UNSUPPORTED,
              "D up to 1024 and up to 65,536 heads together (%d, %d, %d)", d->D, d->H, d->Hkv);
  ROT_REQUIRE(d->width >= 2 && d->width % 2 == 0 && d->width <= d->D, GATTN_ERR_INVALID_ARG,
              "width must be even and from 2 to D (%d, %d)", d->width, d->D);
  ROT_REQUIRE(d->layout == GATTN_ROTARY_HALF || d->layout == GATTN_ROTARY_INTERLEAVED,
              GATTN_ERR_INVALID_ARG, "unknown layout %d", d->layout);
  ROT_REQUIRE(std::isfinite(d->amp), GATTN_ERR_INVALID_ARG, "amp must be finite");
  ROT_REQUIRE(d->pos || d->seq_q || d->S == 0, GATTN_ERR_INVALID_ARG,
              "positions need pos or seq_q (device pointers)");
  ROT_REQUIRE(al(d->pos, 4) && al(d->seq_q, 4) && al(d->seq_k, 4) && al(d->len_k, 4),
              GATTN_ERR_INVALID_ARG, "positions are misaligned");
  const int es = d->dtype == GATTN_F32 ? 4 : 2;
  const int64_t qs = d->q_stride ? d->q_stride : int64_t(d->H) * d->D;
  const int64_t ks = d->k_stride ? d->k_stride : int64_t(d->Hkv) * d->D;
  const int64_t qos = d->q_out_stride ? d->q_out_stride : int64_t(d->H) * d->D;
  const int64_t kos = d->k_out_stride ? d->k_out_stride : int64_t(d->Hkv) * d->D;
  ROT_REQUIRE(d->N <= 1 || (qs >= int64_t(d->H) * d->D && qos >= int64_t(d->H) * d->D &&
                            ks >= int64_t(d->Hkv) * d->D && kos >= int64_t(d->Hkv) * d->D),
              GATTN_ERR_INVALID_ARG, "rows must not overlap: strides of at least heads * D");
  if (d->N == 0 || (d->S == 0 && !d->pos)) return GATTN_OK;
  ROT_REQUIRE(d->freqs && al(d->freqs, 8), GATTN_ERR_INVALID_ARG,
              "freqs must be a device pointer, aligned to 8 bytes");
  ROT_REQUIRE(Q && Q_out && al(Q, es) && al(Q_out, es) &&
                  (d->Hkv == 0 || (K && K_out && al(K, es) && al(K_out, es))),
              GATTN_ERR_INVALID_ARG, "tensors must be non-null device pointers, aligned to elements");
  ROT_REQUIRE((Q != Q_out || qs == qos) && (d->Hkv == 0 || K != K_out || ks == kos),
              GATTN_ERR_INVALID_ARG, "a tensor turned in place keeps its stride");
  RotParams p{};
  p.N = d->N;
  p.H = d->H;
  p.HT = d->H + d->Hkv;
  p.D = d->D;
  p.R = d->width;
  p.S = d->S;
  p.half = d->layout == GATTN_ROTARY_HALF;
  p.amp = d->amp;
  p.sign = d->inverse ? -1.f : 1.f;
  p.freqs = d->freqs;
  p.pos = d->pos;
  p.seq_q = d->seq_q;
  p.seq_k = d->seq_k;
  p.len_k = d->len_k;
  p.q = static_cast<const char*>(Q);
  p.k = static_cast<const char*>(K);
  p.qo = static_cast<char*>(Q_out);
  p.ko = static_cast<char*>(K_out);
  p.qs = qs;
  p.ks = ks;
  p.qos = qos;
  p.kos = kos;
  const int V = 16 / es;
  const auto vec = [&](const void* x, int64_t stride) { return al(x, 16) && stride % V == 0; };
  // vectors: rows and heads start on 16-byte borders; whole: what turns together does too
  const bool vectors = d->D % V == 0 && vec(Q, qs) && vec(Q_out, qos) &&
                       (d->Hkv == 0 || (vec(K, ks) && vec(K_out, kos)));
  const bool whole = vectors && (!p.half || d->width % (2 * V) == 0) && d->D / V <= kRotThreads;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (es == 4) launch<float>(p, vectors, whole, st);
  else launch<__nv_bfloat16>(p, vectors, whole, st);
  const cudaError_t e = cudaGetLastError();
  ROT_REQUIRE(e == cudaSuccess, GATTN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return GATTN_OK;
}

gattn_status gattn_rotary_freqs(int32_t width, double theta, int32_t scaling, double factor,
                                double orig_len, double low, double high, uint64_t* freqs) {
  ROT_REQUIRE(width >= 2 && width % 2 == 0 && width <= 1024, GATTN_ERR_INVALID_ARG,
              "width must be even and from 2 to 1024 (%d)", width);
  ROT_REQUIRE(scaling >= GATTN_ROTARY_PLAIN && scaling <= GATTN_ROTARY_RAMP, GATTN_ERR_INVALID_ARG,
              "unknown scaling %d", scaling);
  ROT_REQUIRE(std::isfinite(theta) && theta >= 1.0, GATTN_ERR_INVALID_ARG,
              "theta must be at least 1");
  ROT_REQUIRE(scaling == GATTN_ROTARY_PLAIN || (std::isfinite(factor) && factor >= 1.0),
              GATTN_ERR_INVALID_ARG, "factor must be at least 1");
  ROT_REQUIRE(scaling != GATTN_ROTARY_RAMP ||
                  (std::isfinite(orig_len) && orig_len > 0.0 && std::isfinite(low) &&
                   std::isfinite(high) && low < high),
              GATTN_ERR_INVALID_ARG, "a ramp needs orig_len > 0 and low < high");
  ROT_REQUIRE(freqs != nullptr, GATTN_ERR_INVALID_ARG, "freqs is NULL");
  constexpr double kTwoPi = 6.283185307179586476925;
  if (scaling == GATTN_ROTARY_BASE && width > 2)
    theta *= std::pow(factor, double(width) / (width - 2));
  for (int i = 0; i < width / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / width);
    if (scaling == GATTN_ROTARY_LINEAR) f /= factor;
    if (scaling == GATTN_ROTARY_RAMP) {
      const double g = std::fmin(std::fmax((orig_len * f / kTwoPi - low) / (high - low), 0.0), 1.0);
      f *= g + (1.0 - g) / factor;
    }
    freqs[i] = uint64_t(std::llrint(std::ldexp(f / kTwoPi, 62))) << 2;  // f <= 1: under 2^60
  }
  return GATTN_OK;
}

}  // extern "C"
