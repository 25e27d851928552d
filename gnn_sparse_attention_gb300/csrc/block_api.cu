// block_api.cu -- C ABI of block selection and block attention, and the small
// kernels around the backward: Delta = dout . out, the transpose of the block
// lists, and the join of split work.
//
// The transpose: bits[block][head][unit] marks which units chose a block
// (atomicOr, so its result does not hang on the order); the units of a
// 128-key tile are the set bits of its blocks in ascending order, cut into
// work items of at most `chunk` units.  A tile with more than one item sums
// its items' fp32 partials in item order.
//
// Measured (65,536 nodes, 8 heads of 64, 16 blocks): Delta 27 us (134 MB, 4.9 TB/s),
// marks, counts and items 18 us, the join 6 us; 24 us where every tile has several
// items (16,384 tokens, 4 key heads of 128).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attn_launch.cuh"
#include "block_items.cuh"
#include "block_tc.cuh"

namespace gattn {

int sm_count() {  // of the current device; asked once per device
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

static std::atomic<int> g_wait_test{0};
int block_wait_test() { return g_wait_test.load(std::memory_order_relaxed); }

namespace {

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

#define BLOCK_REQUIRE(cond, code, ...)   \
  do {                                   \
    if (!(cond)) {                       \
      set_error("gattn_block: " __VA_ARGS__); \
      return code;                       \
    }                                    \
  } while (0)

gattn_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s launch failed: %s", what, cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  return GATTN_OK;
}

gattn_status geom(const gattn_block_desc* d, BlockGeom* g) {
  BLOCK_REQUIRE(d != nullptr, GATTN_ERR_INVALID_ARG, "desc is NULL");
  BLOCK_REQUIRE(d->dtype == GATTN_F32 || d->dtype == GATTN_BF16, GATTN_ERR_INVALID_ARG,
                "unknown dtype %d", d->dtype);
  BLOCK_REQUIRE(d->S >= 0 && d->Nq >= 0 && d->Nk >= 0, GATTN_ERR_INVALID_ARG,
                "S, Nq and Nk must not be negative (%d, %d, %d)", d->S, d->Nq, d->Nk);
  BLOCK_REQUIRE(d->H > 0 && d->Hkv > 0 && d->D > 0 && d->topk > 0, GATTN_ERR_INVALID_ARG,
                "H, Hkv, D and topk must be positive (%d, %d, %d, %d)", d->H, d->Hkv, d->D,
                d->topk);
  const int es = d->dtype == GATTN_F32 ? 4 : 2;
  BLOCK_REQUIRE(pow2(d->D) && d->D * es >= 16 && d->D <= 128 && pow2(d->H) && pow2(d->Hkv) &&
                    d->Hkv <= d->H && d->H / d->Hkv <= 128 && int64_t(d->H) * d->D <= 65536,
                GATTN_ERR_UNSUPPORTED,
                "unsupported heads H=%d Hkv=%d D=%d: need powers of two, Hkv <= H <= 128 Hkv, "
                "16 <= D * size, D <= 128, H * D <= 65536", d->H, d->Hkv, d->D);
  BLOCK_REQUIRE(pow2(d->block) && d->block >= 16 && d->block <= 128 && pow2(d->q_block) &&
                    d->q_block <= 128,
                GATTN_ERR_UNSUPPORTED,
                "block must be 16, 32, 64 or 128 and q_block a power of two up to 128 (%d, %d)",
                d->block, d->q_block);
  BLOCK_REQUIRE(d->topk <= kBlkMaxTopk, GATTN_ERR_UNSUPPORTED, "topk must be at most %d (got %d)",
                kBlkMaxTopk, d->topk);
  BLOCK_REQUIRE(d->scale >= 0.f && std::isfinite(d->scale), GATTN_ERR_INVALID_ARG,
                "scale must be positive (0 for 1/sqrt(D))");
  BLOCK_REQUIRE(d->S == 0 || (d->seq_q && d->seq_k), GATTN_ERR_INVALID_ARG,
                "seq_q and seq_k must be device pointers");
  BLOCK_REQUIRE(al(d->seq_q, 4) && al(d->seq_k, 4) && al(d->len_k, 4), GATTN_ERR_INVALID_ARG,
                "offsets are misaligned");
  BLOCK_REQUIRE(d->max_len_k >= 0, GATTN_ERR_INVALID_ARG, "max_len_k must not be negative");
  g->S = d->S;
  g->Nq = d->Nq;
  g->Nk = d->Nk;
  g->H = d->H;
  g->Hkv = d->Hkv;
  g->G = d->H / d->Hkv;
  g->D = d->D;
  g->block = d->block;
  g->qb = d->q_block;
  g->topk = d->topk;
  g->causal = d->causal != 0;
  g->U = d->S ? d->Nq / d->q_block + (d->q_block > 1 ? d->S : 0) : 0;
  g->B = d->S ? d->Nk / d->block + d->S : 0;
  g->KT = d->S ? d->Nk / kBlkTile + d->S : 0;
  g->scale = d->scale != 0.f ? d->scale : float(1.0 / std::sqrt(double(d->D)));
  g->qmul = g->scale * kLog2e;
  g->seq_q = d->seq_q;
  g->seq_k = d->seq_k;
  g->len_k = d->len_k;
  const bool packed = d->idx_stride[0] == 0 && d->idx_stride[1] == 0;
  BLOCK_REQUIRE(d->idx_stride[0] >= 0 && d->idx_stride[1] >= 0, GATTN_ERR_INVALID_ARG,
                "idx_stride must not be negative");
  g->is_u = packed ? int64_t(d->Hkv) * d->topk : d->idx_stride[0];
  g->is_h = packed ? d->topk : d->idx_stride[1];
  BLOCK_REQUIRE(int64_t(d->Nq) + d->S < INT32_MAX && int64_t(d->Nk) + d->S < INT32_MAX &&
                    int64_t(g->KT) * g->Hkv < INT32_MAX,
                GATTN_ERR_UNSUPPORTED, "too many rows");
  return GATTN_OK;
}

gattn_status check_ws(const char* what, const void* ws, size_t have, size_t need) {
  if (need && (!ws || !al(ws, 16) || have < need)) {
    set_error("%s: workspace needs %zu bytes (16-byte aligned), got %zu", what, need, have);
    return GATTN_ERR_INVALID_ARG;
  }
  return GATTN_OK;
}

gattn_status check_ptrs(const char* what, std::initializer_list<const void*> list) {
  for (const void* p : list)
    if (!p || !al(p, 16)) {
      set_error("%s: tensors must be non-null 16-byte aligned device pointers", what);
      return GATTN_ERR_INVALID_ARG;
    }
  return GATTN_OK;
}

// --------------------------------------------------------------------------
// backward: workspace and preparation
// --------------------------------------------------------------------------
constexpr int64_t kMaxItems = INT32_MAX - 65536;  // every CTA counts one item past the last

BlockBwdWs bwd_ws(const BlockGeom& g, bool f32) {
  BlockBwdWs w{};
  w.words = (g.U + 31) / 32;
  const int64_t entries = int64_t(g.U) * g.Hkv * g.topk;
  w.chunk = item_units(entries, g.qb * g.G, sm_count(), f32);
  w.slots = item_slots(entries, w.chunk);
  w.max_items = int64_t(g.KT) * g.Hkv + w.slots;
  size_t o = 0;
  w.stat = o;
  o = up256(o + size_t(g.Nq) * g.H * 8);
  w.bits = o;
  o += size_t(g.B) * g.Hkv * w.words * 4;
  w.head = o = up256(o);  // cleared together with the bits
  o = up256(o + 16);
  w.cnt = o;
  o = up256(o + size_t(g.KT) * g.Hkv * 8);
  w.items = o;
  o = up256(o + size_t(w.max_items) * 16);
  w.part = o;
  o = up256(o + size_t(w.slots) * 2 * kBlkTile * g.D * 4);
  w.total = o;
  return w;
}

// The backward's statistics of a (row, head): lse log2(e) and Delta = dout . out;
// 16 bytes a lane, D / V lanes a head.
template <class T, int V>
__global__ void __launch_bounds__(256) stat_kernel(const T* __restrict__ o,
                                                    const T* __restrict__ go,
                                                    const float* __restrict__ lse, float2* stat,
                                                    int64_t n, int D) {
  const int tpr = D / V;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  float s = 0.f;
  if (i < n * tpr) {
    const uint4 a = reinterpret_cast<const uint4*>(o)[i], b = reinterpret_cast<const uint4*>(go)[i];
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (V == 4) {
        s = fmaf(__uint_as_float(x[k]), __uint_as_float(y[k]), s);
      } else {
        s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
        s = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), s);
      }
    }
  }
  for (int x = tpr >> 1; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  if (i < n * tpr && threadIdx.x % tpr == 0) stat[i / tpr] = make_float2(lse[i / tpr] * kLog2e, s);
}

// one warp per unit: its bit in every block it lists
__global__ void __launch_bounds__(256) mark_kernel(const BlockBwdParams p) {
  const BlockGeom& g = p.g;
  const int u = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= g.U) return;
  const Unit un = unit_at(g, u);
  if (un.n == 0) return;
  const int nb = (span_k(g, un.s).len + g.block - 1) / g.block;
  const int b0 = piece_base(g.seq_k, un.s, g.block);
  const int32_t* idx = p.idx + int64_t(u) * g.is_u;
  for (int e = threadIdx.x & 31; e < g.Hkv * g.topk; e += 32) {
    const int kh = e / g.topk, b = idx[kh * g.is_h + (e - kh * g.topk)];
    if (b >= 0 && b < nb && b0 + b < g.B)
      atomicOr(p.bits + (int64_t(b0 + b) * g.Hkv + kh) * p.words + (u >> 5), 1u << (u & 31));
  }
}

// one warp per (key tile, head): units that chose one of its blocks
__global__ void __launch_bounds__(256) count_kernel(const BlockBwdParams p) {
  const BlockGeom& g = p.g;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= g.KT * g.Hkv) return;
  const int kt = i / g.Hkv, kh = i - kt * g.Hkv;
  const int s = piece_seq(g.seq_k, g.S, kBlkTile, kt);
  const Span ks = span_k(g, s), qs = span_q(g, s);
  const int64_t pos = int64_t(kt - piece_base(g.seq_k, s, kBlkTile)) * kBlkTile;
  int c = -1;  // a table row that is no key tile
  if (pos >= 0 && pos < ks.len) {
    const int per = kBlkTile / g.block, bl0 = int(pos) / g.block;
    const int nb = min(per, (ks.len + g.block - 1) / g.block - bl0);
    const int brow = min(piece_base(g.seq_k, s, g.block) + bl0, g.B - nb);
    const int ub = piece_base(g.seq_q, s, g.qb), nu = (qs.len + g.qb - 1) / g.qb;
    c = 0;
    if (nu > 0)
      for (int w = ub / 32 + lane; w <= min((ub + nu - 1) / 32, p.words - 1); w += 32) {
        uint32_t any = 0;
        for (int b = 0; b < nb; ++b)
          any |= p.bits[(int64_t(brow + b) * g.Hkv + kh) * p.words + w];
        c += __popc(any);
      }
    c = __reduce_add_sync(0xffffffffu, c);
  }
  if (lane == 0) p.cnt[2 * i] = c;
}

// one CTA: item and slot numbers by a scan over the key tiles, and the items
__global__ void __launch_bounds__(1024) items_kernel(const BlockBwdParams p, int64_t slots) {
  __shared__ int2 sh[32];
  __shared__ longlong2 base;
  const int n = p.g.KT * p.g.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) base = make_longlong2(0, 0);
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int k = i < n ? tile_items(p.cnt[2 * i], p.chunk) : 0;
    int2 v = make_int2(k, k > 1 ? k : 0), x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
      if (lane >= o) {
        x.x += a;
        x.y += b;
      }
    }
    __syncthreads();  // the previous round's reads of sh and base are done
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    longlong2 before = base;
    for (int w = 0; w < warp; ++w) {
      before.x += sh[w].x;
      before.y += sh[w].y;
    }
    put_items(i, k, before.x + x.x - v.x, before.y + x.y - v.y, p.chunk, slots, p.max_items,
              p.cnt + 2 * i, p.items);
    __syncthreads();
    if (threadIdx.x == 1023) base = make_longlong2(before.x + x.x, before.y + x.y);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.head[0] = int(min(static_cast<long long>(base.x), static_cast<long long>(p.max_items)));
    p.head[1] = 0;
  }
}

// dK, dV of the key tiles with several items: the sums of their partials.
// Most tiles have one, so a warp looks at 32 of a CTA's tiles at a time (a CTA
// for each tile took 37 us at 64k nodes).  A tile that most units chose may have a
// hundred partials: its elements are spread over gridDim.y CTAs.
template <class T>
__global__ void __launch_bounds__(256) join_kv_kernel(const BlockBwdParams p) {
  const BlockGeom& g = p.g;
  const int D = g.D, tiles = g.KT * g.Hkv, lane = threadIdx.x & 31;
  for (int64_t base = blockIdx.x; base < tiles; base += int64_t(gridDim.x) * 32) {
    const int64_t mine = base + int64_t(lane) * gridDim.x;
    const int2 own = mine < tiles ? reinterpret_cast<const int2*>(p.cnt)[mine] : make_int2(0, 0);
    for (unsigned m = __ballot_sync(0xffffffffu, own.x > p.chunk); m; m &= m - 1) {
      const int b = __ffs(m) - 1, i = int(base + int64_t(b) * gridDim.x);
      const int c = __shfl_sync(0xffffffffu, own.x, b);
      const int kt = i / g.Hkv, kh = i - kt * g.Hkv;
      const int s = piece_seq(g.seq_k, g.S, kBlkTile, kt);
      const Span ks = span_k(g, s);
      const int pos = (kt - piece_base(g.seq_k, s, kBlkTile)) * kBlkTile;
      const int n = (c + p.chunk - 1) / p.chunk;
      const float* part =
          p.part + int64_t(__shfl_sync(0xffffffffu, own.y, b)) * 2 * kBlkTile * D;
      for (int e = (threadIdx.x + blockIdx.y * 256) * 4; e < 2 * kBlkTile * D;
           e += 1024 * gridDim.y) {
        const int which = e / (kBlkTile * D), r = (e / D) % kBlkTile, d = e % D;
        if (pos + r >= ks.len) continue;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
          const float4 x =
              *reinterpret_cast<const float4*>(part + int64_t(k) * 2 * kBlkTile * D + e);
          t.x += x.x;
          t.y += x.y;
          t.z += x.z;
          t.w += x.w;
        }
        const float mul = which ? 1.f : g.scale;
        T* out =
            static_cast<T*>(which ? p.dV : p.dK) + (int64_t(ks.beg + pos + r) * g.Hkv + kh) * D + d;
        out[0] = T(t.x * mul);
        out[1] = T(t.y * mul);
        out[2] = T(t.z * mul);
        out[3] = T(t.w * mul);
      }
    }
  }
}

gattn_status bwd_prepare(const BlockBwdParams& p, gattn_dtype dt, const BlockBwdWs& w, char* ws,
                         cudaStream_t st) {
  const BlockGeom& g = p.g;
  if (cudaMemsetAsync(ws + w.bits, 0, w.head + 16 - w.bits, st) != cudaSuccess) {
    set_error("gattn_block_bwd: clearing the workspace failed");
    return GATTN_ERR_CUDA;
  }
  const int64_t n = int64_t(g.Nq) * g.H;
  const int V = dt == GATTN_F32 ? 4 : 8;
  const unsigned grid = unsigned((n * (g.D / V) + 255) / 256);
  if (n > 0 && dt == GATTN_F32)
    stat_kernel<float, 4><<<grid, 256, 0, st>>>(static_cast<const float*>(p.O),
                                                 static_cast<const float*>(p.dO), p.lse, p.stat, n,
                                                 g.D);
  else if (n > 0)
    stat_kernel<__nv_bfloat16, 8><<<grid, 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(p.O), static_cast<const __nv_bfloat16*>(p.dO), p.lse,
        p.stat, n, g.D);
  if (g.U > 0) mark_kernel<<<(g.U + 7) / 8, 256, 0, st>>>(p);
  count_kernel<<<(g.KT * g.Hkv + 7) / 8, 256, 0, st>>>(p);
  items_kernel<<<1, 1024, 0, st>>>(p, w.slots);
  return launched("gattn_block_bwd (preparation)");
}

}  // namespace

}  // namespace gattn

using namespace gattn;

extern "C" {

gattn_status gattn_block_sums(const gattn_block_desc* desc, const void* K, const int32_t* since,
                              double* sums, gattn_stream_t stream) {
  BlockGeom g{};
  gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  if (g.B == 0) return GATTN_OK;
  if ((g.Nk > 0 && (s = check_ptrs("gattn_block_sums", {K})) != GATTN_OK) ||
      (s = check_ptrs("gattn_block_sums", {sums})) != GATTN_OK)
    return s;
  BLOCK_REQUIRE(al(since, 4), GATTN_ERR_INVALID_ARG, "since is misaligned");
  return launch_block_sums(g, gattn_dtype(desc->dtype), K, false, since, sums,
                           reinterpret_cast<cudaStream_t>(stream));
}

// 64-bit sums of the units' queries (single-row units are summed on the fly)
static size_t select_ws(const BlockGeom& g) {
  return g.qb == 1 ? 0 : size_t(g.U) * g.Hkv * g.D * 8;
}

gattn_status gattn_block_select_workspace_size(const gattn_block_desc* desc, size_t* bytes) {
  BlockGeom g{};
  const gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  BLOCK_REQUIRE(bytes, GATTN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = select_ws(g);
  return GATTN_OK;
}

gattn_status gattn_block_select(const gattn_block_desc* desc, const void* Q, const double* sums,
                                int32_t* idx, void* workspace, size_t workspace_bytes,
                                gattn_stream_t stream) {
  BlockGeom g{};
  gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  if (g.U == 0) return GATTN_OK;
  if ((s = check_ptrs("gattn_block_select", {sums})) != GATTN_OK ||
      (g.Nq > 0 && (s = check_ptrs("gattn_block_select", {Q})) != GATTN_OK) ||
      (s = check_ws("gattn_block_select", workspace, workspace_bytes, select_ws(g))) != GATTN_OK)
    return s;
  BLOCK_REQUIRE(idx && al(idx, 4), GATTN_ERR_INVALID_ARG, "idx must be a device pointer");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const gattn_dtype dt = gattn_dtype(desc->dtype);
  double* qsum = g.qb == 1 ? nullptr : static_cast<double*>(workspace);
  if (qsum && (s = launch_block_sums(g, dt, Q, true, nullptr, qsum, st)) != GATTN_OK) return s;
  const int64_t len = desc->max_len_k > 0 ? std::min(desc->max_len_k, g.Nk) : g.Nk;
  return launch_block_select(g, dt, Q, qsum, sums, int((len + g.block - 1) / g.block), idx, st);
}

gattn_status gattn_block_fwd_workspace_size(const gattn_block_desc* desc, size_t* bytes) {
  BlockGeom g{};
  const gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  BLOCK_REQUIRE(bytes, GATTN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = desc->dtype == GATTN_BF16 && g.U > 0 ? block_fwd_tc_workspace(g) : 0;
  return GATTN_OK;
}

gattn_status gattn_block_fwd(const gattn_block_desc* desc, const void* Q, const void* K,
                             const void* V, const int32_t* idx, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, gattn_stream_t stream) {
  BlockGeom g{};
  gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  if (g.U == 0 || g.Nq == 0) return GATTN_OK;
  if ((s = check_ptrs("gattn_block_fwd", {Q, out})) != GATTN_OK ||
      (g.Nk > 0 && (s = check_ptrs("gattn_block_fwd", {K, V})) != GATTN_OK))
    return s;
  BLOCK_REQUIRE(idx && al(idx, 4) && lse && al(lse, 4), GATTN_ERR_INVALID_ARG,
                "idx and lse must be device pointers");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (desc->dtype == GATTN_F32)
    return launch_block_fwd_simt(g, static_cast<const float*>(Q), static_cast<const float*>(K),
                                 static_cast<const float*>(V), idx, static_cast<float*>(out), lse,
                                 st);
  if ((s = check_ws("gattn_block_fwd", workspace, workspace_bytes, block_fwd_tc_workspace(g))) !=
      GATTN_OK)
    return s;
  return launch_block_fwd_tc(g, Q, K, V, idx, out, lse, workspace, st);
}

gattn_status gattn_block_bwd_workspace_size(const gattn_block_desc* desc, size_t* bytes) {
  BlockGeom g{};
  const gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  BLOCK_REQUIRE(bytes, GATTN_ERR_INVALID_ARG, "bytes is NULL");
  const BlockBwdWs w = bwd_ws(g, desc->dtype == GATTN_F32);
  BLOCK_REQUIRE(w.max_items < kMaxItems, GATTN_ERR_UNSUPPORTED, "too many rows");
  *bytes = w.total;
  return GATTN_OK;
}

gattn_status gattn_block_bwd(const gattn_block_desc* desc, const void* Q, const void* K,
                             const void* V, const int32_t* idx, const void* out, const void* dout,
                             const float* lse, void* dQ, void* dK, void* dV, void* workspace,
                             size_t workspace_bytes, gattn_stream_t stream) {
  BlockGeom g{};
  gattn_status s = geom(desc, &g);
  if (s != GATTN_OK) return s;
  if (g.S == 0 || (g.Nq == 0 && g.Nk == 0)) return GATTN_OK;
  const BlockBwdWs w = bwd_ws(g, desc->dtype == GATTN_F32);
  BLOCK_REQUIRE(w.max_items < kMaxItems, GATTN_ERR_UNSUPPORTED, "too many rows");
  if ((g.Nq > 0 && (s = check_ptrs("gattn_block_bwd", {Q, out, dout, dQ})) != GATTN_OK) ||
      (g.Nk > 0 && (s = check_ptrs("gattn_block_bwd", {K, V, dK, dV})) != GATTN_OK) ||
      (s = check_ws("gattn_block_bwd", workspace, workspace_bytes, w.total)) != GATTN_OK)
    return s;
  BLOCK_REQUIRE(g.Nq == 0 || (idx && al(idx, 4) && lse && al(lse, 4)), GATTN_ERR_INVALID_ARG,
                "idx and lse must be device pointers");
  char* ws = static_cast<char*>(workspace);
  BlockBwdParams p{};
  p.g = g;
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.O = out;
  p.dO = dout;
  p.idx = idx;
  p.lse = lse;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  p.stat = reinterpret_cast<float2*>(ws + w.stat);
  p.bits = reinterpret_cast<uint32_t*>(ws + w.bits);
  p.head = reinterpret_cast<int32_t*>(ws + w.head);
  p.cnt = reinterpret_cast<int32_t*>(ws + w.cnt);
  p.items = reinterpret_cast<int4*>(ws + w.items);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.words = w.words;
  p.chunk = w.chunk;
  p.max_items = w.max_items;
  p.fail = block_wait_test();
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const gattn_dtype dt = gattn_dtype(desc->dtype);
  if ((s = bwd_prepare(p, dt, w, ws, st)) != GATTN_OK ||
      (s = dt == GATTN_F32 ? launch_block_bwd_simt(p, st) : launch_block_bwd_tc(p, st)) !=
          GATTN_OK)
    return s;
  const dim3 grid(std::min(g.KT * g.Hkv, 2 * sm_count()), std::max(1, kBlkTile * g.D * 2 / 1024));
  if (dt == GATTN_F32) join_kv_kernel<float><<<grid, 256, 0, st>>>(p);
  else join_kv_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  return launched("gattn_block_bwd (join)");
}

gattn_status gattn_block_set_wait_test(int32_t fail_first_wait) {
  g_wait_test.store(fail_first_wait != 0, std::memory_order_relaxed);
  return GATTN_OK;
}

gattn_status gattn_block_check_errors(void) {
  cudaError_t e = cudaDeviceSynchronize();
  int fwd = 0, bwd = 0;
  if (e == cudaSuccess) e = block_fwd_tc_take_error(&fwd);
  if (e == cudaSuccess) e = block_bwd_tc_take_error(&bwd);
  if (e != cudaSuccess) {
    set_error("gattn_block_check_errors: %s", cudaGetErrorString(e));
    return GATTN_ERR_CUDA;
  }
  if (fwd || bwd) {
    set_error("a block-attention kernel gave up a bounded wait");
    return GATTN_ERR_TIMEOUT;
  }
  return GATTN_OK;
}

}  // extern "C"
