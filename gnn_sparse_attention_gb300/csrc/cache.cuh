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
// that sequence; s = -1 for none.  Every lane searches for a row of its own.  With one
// row a sequence, as in serving, row r is sequence r: looked at first, since a search is
// a chain of loads.
struct SeqRow {
  int s, i, n;
};
__device__ __forceinline__ SeqRow seq_row(const int32_t* __restrict__ beg, int S, int N, int r) {
  if (S <= 0) return {-1, 0, 0};
  int lo = min(r, S - 1), b = beg[lo], e = beg[lo + 1];
  if (r < b || r >= e) {
    lo = 0;  // the last s with beg[s] <= r, if beg[0] is one
    for (int hi = S; hi - lo > 1;) {
      const int mid = lo + (hi - lo) / 2;
      if (beg[mid] <= r) lo = mid;
      else hi = mid;
    }
    b = beg[lo];
    e = beg[lo + 1];
  }
  b = clampi(b, 0, N);
  const int n = clampi(e, b, N) - b, i = r - b;
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
