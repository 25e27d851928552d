// block.cuh -- shapes and device lookups shared by the block-selection and
// block-attention kernels (block_*.cu).
//
// Pieces.  Sequence s is cut into pieces of `per` rows; piece j of it has the
// table row base(s) + j, base(s) = beg[s] / per + s (+ 0 for one-row pieces).
// ceil(len / per) <= (end / per - beg / per) + 1 keeps the sequences' table
// rows apart for any offsets, so tables are sized and addressed without
// reading a length on the host.
#pragma once

#include "gattn_internal.cuh"

namespace gattn {

constexpr int kBlkTile = 128;     // keys per step, rows per tile
constexpr int kBlkMaxTopk = 128;

struct BlockGeom {
  int S, Nq, Nk, H, Hkv, G, D;
  int block, qb, topk, causal;
  int U, B;          // units, blocks (table rows)
  int KT;            // 128-key tiles (table rows)
  float qmul, scale;  // scale * log2(e), scale
  const int32_t *seq_q, *seq_k, *len_k;
  int64_t is_u, is_h;  // strides of idx
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

struct Span {
  int beg, len;
};
// rows of sequence s, cut to the tensors whatever the offsets say
__device__ __forceinline__ Span span_q(const BlockGeom& g, int s) {
  const int b = clampi(g.seq_q[s], 0, g.Nq);
  return {b, clampi(g.seq_q[s + 1], b, g.Nq) - b};
}
__device__ __forceinline__ Span span_k(const BlockGeom& g, int s) {
  const int b = clampi(g.seq_k[s], 0, g.Nk);
  const int room = clampi(g.seq_k[s + 1], b, g.Nk) - b;
  return {b, g.len_k ? clampi(g.len_k[s], 0, room) : room};
}

// Sequence whose pieces include table row `row`: the last s with base(s) <=
// row, found by the 32 lanes of a warp (all call it; same result in all).
__device__ __forceinline__ int piece_seq(const int32_t* beg, int S, int per, int row) {
  const int lane = threadIdx.x & 31, one = per > 1 ? 1 : 0;
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < lo + n && max(beg[i], 0) / per + one * i <= row;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int hi = m ? 31 - __clz(m) : 0;
    n = min(step, n - hi * step);
    lo += hi * step;
  }
  return lo;
}
__device__ __forceinline__ int piece_base(const int32_t* beg, int s, int per) {
  return max(beg[s], 0) / per + (per > 1 ? s : 0);
}

// Unit `u`: its sequence, first row, rows (0 when the table row belongs to
// nothing) and the position of its first row.
struct Unit {
  int s, row, n, pos;
};
__device__ __forceinline__ Unit unit_at(const BlockGeom& g, int u) {
  Unit x;
  x.s = piece_seq(g.seq_q, g.S, g.qb, u);
  const Span q = span_q(g, x.s);
  const int64_t off = int64_t(u - piece_base(g.seq_q, x.s, g.qb)) * g.qb;
  const bool in = off >= 0 && off < q.len;
  x.row = in ? q.beg + int(off) : 0;
  x.n = in ? min(g.qb, q.len - int(off)) : 0;
  x.pos = in ? int(off) + span_k(g, x.s).len - q.len : 0;
  return x;
}

// The entries of one idx row that name something, sorted and without
// repeats: one warp reads idx[0, topk), writes ids[0, n) (shared memory) and
// returns n.  `nb` blocks belong to the sequence.
__device__ __forceinline__ int block_list(const int32_t* idx, int topk, int nb, int* ids) {
  const int lane = threadIdx.x & 31;
  int v[kBlkMaxTopk / 32];
  bool ok[kBlkMaxTopk / 32];
  bool sorted = true;  // strictly ascending, nothings last
  int last = -1, n = 0;
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c) {
    const int e = c * 32 + lane;
    v[c] = e < topk ? idx[e] : -1;
    ok[c] = v[c] >= 0 && v[c] < nb;
    const int prev = __shfl_up_sync(0xffffffffu, v[c], 1);
    const unsigned m = __ballot_sync(0xffffffffu, ok[c]);
    const bool here = !ok[c] || (lane == 0 ? v[c] > last : v[c] > prev);
    sorted = sorted && (m & (m + 1)) == 0 && (m == 0 || n == c * 32) &&
             __all_sync(0xffffffffu, here);
    n += __popc(m);
    last = __shfl_sync(0xffffffffu, v[c], 31);
  }
  if (sorted) {
#pragma unroll
    for (int c = 0; c < kBlkMaxTopk / 32; ++c)
      if (ok[c]) ids[c * 32 + lane] = v[c];
    __syncwarp();
    return n;
  }
  // rank among the valid entries: smaller ids, first occurrences only
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c) ids[c * 32 + lane] = ok[c] ? v[c] : -1;
  __syncwarp();
  int rank[kBlkMaxTopk / 32];
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c) {
    bool first = ok[c];
    for (int e = 0; e < c * 32 + lane; ++e) first = first && ids[e] != v[c];
    ok[c] = first;
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c) ids[c * 32 + lane] = ok[c] ? v[c] : INT32_MAX;
  __syncwarp();
  n = 0;
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c) {
    int r = 0;
    if (ok[c])
      for (int e = 0; e < kBlkMaxTopk; ++e) r += ids[e] < v[c];
    rank[c] = r;
    n += __popc(__ballot_sync(0xffffffffu, ok[c]));
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kBlkMaxTopk / 32; ++c)
    if (ok[c]) ids[rank[c]] = v[c];
  __syncwarp();
  return n;
}

// Keys of the sorted list at positions below `end`: with the list ascending
// these are the first columns of the steps, so a row's mask is one number.
__device__ __forceinline__ int list_keys(const int* ids, int n, int block, int end) {
  int lo = 0, hi = n;  // ids[0, lo) start below end
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (ids[mid] * block < end) lo = mid + 1;
    else hi = mid;
  }
  return lo == 0 ? 0 : (lo - 1) * block + min(block, end - ids[lo - 1] * block);
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------
// A unit's (query row, head) pairs of one key head as 128-row tiles: `ht`
// heads by qb rows each.
inline int tile_heads(const BlockGeom& g) { return g.G < kBlkTile / g.qb ? g.G : kBlkTile / g.qb; }

// Workspace of the backward (byte offsets).
struct BlockBwdWs {
  size_t stat, bits, head, cnt, items, part, total;
  int words;         // 32-bit words of a bitmap row (units)
  int chunk;         // units per work item
  int64_t max_items, slots;
};

struct BlockBwdParams {
  BlockGeom g;
  const void *Q, *K, *V, *O, *dO;
  const int32_t* idx;
  const float* lse;
  void *dQ, *dK, *dV;
  float2* stat;      // [Nq][H]: lse log2(e), Delta
  uint32_t* bits;    // [B][Hkv][words]: units that chose the block
  int32_t* head;     // [4]: items, next item, slots
  int32_t* cnt;      // [KT * Hkv][2]: units of the key tile, first partial slot
  int4* items;       // (key tile * Hkv + head, first unit, units, slot or -1)
  float* part;       // [slots][2][128][D]: dK, dV of one item
  int words, chunk;
  int fail;          // failure-path test: the compute warps give up their first wait
  int64_t max_items;
};

int sm_count();
int block_wait_test();  // what gattn_block_set_wait_test set
gattn_status launch_block_fwd_simt(const BlockGeom& g, const float* Q, const float* K,
                                   const float* V, const int32_t* idx, float* out, float* lse,
                                   cudaStream_t st);
gattn_status launch_block_bwd_simt(const BlockBwdParams& p, cudaStream_t st);
gattn_status launch_block_sums(const BlockGeom& g, gattn_dtype dt, const void* x, bool queries,
                               const int32_t* since, double* sums, cudaStream_t st);
gattn_status launch_block_select(const BlockGeom& g, gattn_dtype dt, const void* Q,
                                 const double* qsum, const double* sums, int max_blocks,
                                 int32_t* idx, cudaStream_t st);

}  // namespace gattn
