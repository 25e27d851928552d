// cache_api.cu -- C ABI of the quantised key/value cache: checks on the host.
#include <algorithm>
#include <cmath>

#include "cache.cuh"

namespace gattn {

namespace {

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

#define CACHE_REQUIRE(cond, code, ...)        \
  do {                                        \
    if (!(cond)) {                            \
      set_error("gattn_cache: " __VA_ARGS__); \
      return code;                            \
    }                                         \
  } while (0)

enum Use { kRows, kSums, kAttention };

gattn_status params(const gattn_cache_desc* d, Use use, CacheParams* p) {
  CACHE_REQUIRE(d != nullptr, GATTN_ERR_INVALID_ARG, "desc is NULL");
  CACHE_REQUIRE(d->dtype == GATTN_F32 || d->dtype == GATTN_BF16, GATTN_ERR_INVALID_ARG,
                "unknown dtype %d", d->dtype);
  CACHE_REQUIRE(d->S >= 0 && d->N >= 0 && d->Nk >= 0, GATTN_ERR_INVALID_ARG,
                "S, N and Nk must not be negative (%d, %d, %d)", d->S, d->N, d->Nk);
  CACHE_REQUIRE(d->bits == 4 || d->bits == 8, GATTN_ERR_UNSUPPORTED, "bits must be 4 or 8 (got %d)",
                d->bits);
  CACHE_REQUIRE(d->D == 32 || d->D == 64 || d->D == 128, GATTN_ERR_UNSUPPORTED,
                "D must be 32, 64 or 128 (got %d)", d->D);
  CACHE_REQUIRE(pow2(d->Hkv) && d->Hkv <= 1024, GATTN_ERR_UNSUPPORTED,
                "Hkv must be a power of two up to 1024 (got %d)", d->Hkv);
  // the attention counts rows a few steps beyond the last in 32 bits
  CACHE_REQUIRE(int64_t(d->N) + d->S < INT32_MAX && int64_t(d->Nk) + d->S < INT32_MAX - 65536 &&
                    int64_t(d->N) * d->Hkv < (int64_t(1) << 33) &&
                    int64_t(d->Nk) * d->Hkv < (int64_t(1) << 33),
                GATTN_ERR_UNSUPPORTED, "too many rows");
  const bool q = use != kSums;
  CACHE_REQUIRE(d->S == 0 || ((d->seq_q || !q) && d->seq_k), GATTN_ERR_INVALID_ARG,
                "seq_q and seq_k must be device pointers");
  CACHE_REQUIRE(al(d->seq_q, 4) && al(d->seq_k, 4) && al(d->len_k, 4), GATTN_ERR_INVALID_ARG,
                "offsets are misaligned");
  CACHE_REQUIRE(d->S == 0 || d->Nk == 0 ||
                    (d->k && d->v && d->par && al(d->k, 16) && al(d->v, 16) && al(d->par, 16)),
                GATTN_ERR_INVALID_ARG, "k, v and par must be non-null 16-byte aligned device pointers");
  BlockGeom& g = p->g;
  g = BlockGeom{};
  g.S = d->S;
  g.Nq = d->N;
  g.Nk = d->Nk;
  g.H = g.Hkv = d->Hkv;
  g.G = 1;
  g.D = d->D;
  g.qb = 1;
  g.block = 64;
  g.seq_q = d->seq_q;
  g.seq_k = d->seq_k;
  g.len_k = d->len_k;
  g.U = d->S ? d->N : 0;
  p->bits = d->bits;
  p->k = static_cast<uint8_t*>(d->k);
  p->v = static_cast<uint8_t*>(d->v);
  p->par = static_cast<uint2*>(d->par);
  p->ks = d->row_stride[0] ? d->row_stride[0] : int64_t(d->Hkv) * d->D;
  p->vs = d->row_stride[1] ? d->row_stride[1] : int64_t(d->Hkv) * d->D;
  if (use == kRows) return GATTN_OK;
  CACHE_REQUIRE(pow2(d->block) && d->block >= 16 && d->block <= 128, GATTN_ERR_UNSUPPORTED,
                "block must be 16, 32, 64 or 128 (%d)", d->block);
  g.block = d->block;
  g.B = d->S ? d->Nk / d->block + d->S : 0;
  if (use == kSums) return GATTN_OK;
  CACHE_REQUIRE(pow2(d->H) && d->Hkv <= d->H && d->H / d->Hkv <= 128 &&
                    int64_t(d->H) * d->D <= 65536,
                GATTN_ERR_UNSUPPORTED,
                "unsupported heads H=%d Hkv=%d D=%d: need powers of two, Hkv <= H <= 128 Hkv, "
                "H * D <= 65536", d->H, d->Hkv, d->D);
  CACHE_REQUIRE(d->topk >= 0 && d->topk <= kBlkMaxTopk, GATTN_ERR_UNSUPPORTED,
                "topk must be at most %d (got %d)", kBlkMaxTopk, d->topk);
  CACHE_REQUIRE(d->scale >= 0.f && std::isfinite(d->scale), GATTN_ERR_INVALID_ARG,
                "scale must be positive (0 for 1/sqrt(D))");
  CACHE_REQUIRE(d->max_len_k >= 0, GATTN_ERR_INVALID_ARG, "max_len_k must not be negative");
  CACHE_REQUIRE(d->idx_stride[0] >= 0 && d->idx_stride[1] >= 0, GATTN_ERR_INVALID_ARG,
                "idx_stride must not be negative");
  CACHE_REQUIRE(int64_t(d->N) * d->H <= (int64_t(1) << 30), GATTN_ERR_UNSUPPORTED,
                "N * H must be at most 2^30");
  g.H = d->H;
  g.G = d->H / d->Hkv;
  g.topk = d->topk;
  g.causal = d->causal != 0;
  g.scale = d->scale != 0.f ? d->scale : float(1.0 / std::sqrt(double(d->D)));
  g.qmul = g.scale * kLog2e;
  const bool packed = d->idx_stride[0] == 0 && d->idx_stride[1] == 0;
  g.is_u = packed ? int64_t(d->Hkv) * d->topk : d->idx_stride[0];
  g.is_h = packed ? d->topk : d->idx_stride[1];
  return GATTN_OK;
}

int max_keys(const gattn_cache_desc* d) {
  return d->max_len_k > 0 ? std::min(d->max_len_k, d->Nk) : d->Nk;
}

}  // namespace

}  // namespace gattn

using namespace gattn;

extern "C" {

gattn_status gattn_cache_write(const gattn_cache_desc* desc, const void* K, const void* V,
                               gattn_stream_t stream) {
  CacheParams p{};
  const gattn_status s = params(desc, kRows, &p);
  if (s != GATTN_OK) return s;
  if (p.g.U == 0 || p.g.Nk == 0) return GATTN_OK;
  const int vec = desc->dtype == GATTN_F32 ? 4 : 8, row = desc->Hkv * desc->D;
  CACHE_REQUIRE(K && V && al(K, 16) && al(V, 16), GATTN_ERR_INVALID_ARG,
                "K and V must be non-null 16-byte aligned device pointers");
  CACHE_REQUIRE(desc->N <= 1 || (p.ks >= row && p.vs >= row && p.ks % vec == 0 && p.vs % vec == 0),
                GATTN_ERR_INVALID_ARG,
                "row_stride must be at least Hkv * D and a multiple of 16 bytes");
  return launch_cache_write(p, gattn_dtype(desc->dtype), K, V,
                            reinterpret_cast<cudaStream_t>(stream));
}

gattn_status gattn_cache_read(const gattn_cache_desc* desc, const int32_t* since, void* K, void* V,
                              gattn_stream_t stream) {
  CacheParams p{};
  const gattn_status s = params(desc, kRows, &p);
  if (s != GATTN_OK) return s;
  if (p.g.U == 0 || p.g.Nk == 0 || (!K && !V)) return GATTN_OK;
  CACHE_REQUIRE(al(K, 16) && al(V, 16) && al(since, 4), GATTN_ERR_INVALID_ARG,
                "K and V must be 16-byte aligned device pointers");
  return launch_cache_read(p, gattn_dtype(desc->dtype), since, K, V,
                           reinterpret_cast<cudaStream_t>(stream));
}

gattn_status gattn_cache_sums(const gattn_cache_desc* desc, const int32_t* since, double* sums,
                              gattn_stream_t stream) {
  CacheParams p{};
  const gattn_status s = params(desc, kSums, &p);
  if (s != GATTN_OK) return s;
  if (p.g.B == 0) return GATTN_OK;
  CACHE_REQUIRE(sums && al(sums, 16) && al(since, 4), GATTN_ERR_INVALID_ARG,
                "sums must be a non-null 16-byte aligned device pointer");
  return launch_cache_sums(p, since, sums, reinterpret_cast<cudaStream_t>(stream));
}

gattn_status gattn_cache_fwd_workspace_size(const gattn_cache_desc* desc, size_t* bytes) {
  CacheParams p{};
  const gattn_status s = params(desc, kAttention, &p);
  if (s != GATTN_OK) return s;
  CACHE_REQUIRE(bytes, GATTN_ERR_INVALID_ARG, "bytes is NULL");
  // a list may be given or not: room for either
  *bytes = p.g.U == 0 ? 0
                      : std::max(cache_fwd_workspace(p, gattn_dtype(desc->dtype), max_keys(desc), true),
                                 cache_fwd_workspace(p, gattn_dtype(desc->dtype), max_keys(desc), false));
  return GATTN_OK;
}

gattn_status gattn_cache_fwd(const gattn_cache_desc* desc, const void* Q, const int32_t* idx,
                             void* out, float* lse, void* workspace, size_t workspace_bytes,
                             gattn_stream_t stream) {
  CacheParams p{};
  const gattn_status s = params(desc, kAttention, &p);
  if (s != GATTN_OK) return s;
  if (p.g.U == 0) return GATTN_OK;
  CACHE_REQUIRE(Q && out && al(Q, 16) && al(out, 16) && lse && al(lse, 4), GATTN_ERR_INVALID_ARG,
                "Q and out must be non-null 16-byte aligned device pointers, lse one too");
  CACHE_REQUIRE(al(idx, 4) && (!idx || desc->topk > 0), GATTN_ERR_INVALID_ARG,
                "idx must be a device pointer to lists of topk > 0 entries, or NULL");
  const gattn_dtype dt = gattn_dtype(desc->dtype);
  const size_t need = cache_fwd_workspace(p, dt, max_keys(desc), idx != nullptr);
  if (need && (!workspace || !al(workspace, 16) || workspace_bytes < need)) {
    set_error("gattn_cache_fwd: workspace needs %zu bytes (16-byte aligned), got %zu", need,
              workspace_bytes);
    return GATTN_ERR_INVALID_ARG;
  }
  return launch_cache_fwd(p, dt, max_keys(desc), Q, idx, out, lse, workspace,
                          reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
