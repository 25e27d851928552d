// cache.cuh -- the quantised key/value cache: its format, and where the rows of
// a sequence lie (cache_api.cu, cache_rows.cu, cache_attn.cu, rotary.cu).
#pragma once

#include "block.cuh"

namespace gattn {

struct CacheParams {
  BlockGeom g;  // q_block 1: every row of Q is a unit
  int bits;
  int64_t ks, vs;  // elements between rows of K and of V (write)
  uint8_t *k, *v;
  uint2* par;      // bf16 (m, s) of K, (m, s) of V
};

// The sequence that row `r` belongs to, its number within and the rows of
// that sequence; s = -1 for none.  Every lane searches for a row of its own.
struct SeqRow {
  int s, i, n;
};
__device__ __forceinline__ SeqRow seq_row(const int32_t* __restrict__ beg, int S, int N, int r,
                                          int from = 0) {
  int lo = from, hi = S;  // the last s with beg[s] <= r, if beg[from] is one
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (beg[mid] <= r) lo = mid;
    else hi = mid;
  }
  if (lo >= S) return {-1, 0, 0};
  const int b = clampi(beg[lo], 0, N), n = clampi(beg[lo + 1], b, N) - b;
  const int i = r - b;
  return {i >= 0 && i < n ? lo : -1, i, n};
}

gattn_status launch_cache_write(const CacheParams& p, gattn_dtype dt, const void* K, const void* V,
                                cudaStream_t st);
gattn_status launch_cache_read(const CacheParams& p, gattn_dtype dt, const int32_t* since, void* K,
                               void* V, cudaStream_t st);
gattn_status launch_cache_sums(const CacheParams& p, const int32_t* since, double* sums,
                               cudaStream_t st);
size_t cache_fwd_workspace(const CacheParams& p, gattn_dtype dt, int max_keys, bool lists);
gattn_status launch_cache_fwd(const CacheParams& p, gattn_dtype dt, int max_keys, const void* Q,
                              const int32_t* idx, void* out, float* lse, void* ws, cudaStream_t st);

}  // namespace gattn
